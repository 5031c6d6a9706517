"""The sizes at which the MXFP4 calls say MQ_ERR_UNSUPPORTED, as the header
states them (no GPU: refused before anything is launched)."""
import ctypes

import nested_bit_weight_b200 as mq

FAKE = 0x10000
UNSUPPORTED = 2
ROWS = (1 << 31) - 256                       # the most rows of a matrix


def test_quantize():
    # 2^31 - 256 rows: 2^29 - 64 steps of four rows (fp32: 2^30 - 128 of two)
    for dtype, K in ((0, 2080), (1, 2080), (2, 1056)):
        assert mq.lib.mq_mx4_quantize(FAKE, dtype, ROWS, K, K, FAKE, FAKE, None) == UNSUPPORTED
        assert ROWS * K > 2 ** (40 if dtype == 2 else 41)


def test_dequantize():
    m = mq.MqMx4(FAKE, FAKE, ROWS, 2080)
    for dtype in (0, 2):
        assert mq.lib.mq_mx4_dequantize(ctypes.byref(m), FAKE, dtype, 2080, None) == UNSUPPORTED


def test_from_nested():
    w = mq.MqWeights(FAKE, FAKE, ROWS, 129 * 128, 128, 4)          # (2^24 - 2) x 129 blocks
    assert mq.lib.mq_mx4_from_nested(ctypes.byref(w), FAKE, FAKE, None) == UNSUPPORTED


def test_gemm_bf16():
    M, K = 1 << 27, 4128                                           # 17 steps of 256 columns
    w = mq.MqMx4(FAKE, FAKE, 8, K)
    need = mq.mq_mx4_gemm_bf16_workspace_bytes(M, 8, K)
    assert need > 0
    assert mq.lib.mq_mx4_gemm_bf16(FAKE, M, K, ctypes.byref(w), FAKE, 0, 8, FAKE, need, None) == UNSUPPORTED
