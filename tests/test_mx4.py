"""The MXFP4 entry points without a GPU: sizes, and every refusal before
anything is launched (status, reason)."""
import ctypes

import pytest

import nested_bit_weight_b200 as mq

FAKE = 0x10000          # an aligned address; these calls fail before any access
INVALID, MISALIGNED, WORKSPACE = 1, 3, 6


def test_sizes():
    assert mq.mq_mx4_code_bytes(3, 96) == 3 * 48
    assert mq.mq_mx4_scale_bytes(3, 96) == 512                    # one partial block
    assert mq.mq_mx4_scale_bytes(129, 160) == 2 * 2 * 512
    assert mq.mq_mx4_code_bytes(14336, 4096) == 14336 * 2048
    assert mq.mq_mx4_scale_bytes(14336, 4096) == 14336 * 4096 // 32
    assert mq.mq_mx4_code_bytes(70000, 65536) == 70000 * 32768    # beyond 32 bits
    for rows, K in ((-1, 32), (1, 0), (1, 16), (1, 48), (1 << 31, 32), (1, 1 << 31), (0, 32)):
        assert mq.mq_mx4_code_bytes(rows, K) == 0
        assert mq.mq_mx4_scale_bytes(rows, K) == 0
    # rows cut inside the product need none; others eight rows of codes and scales
    # for each row of X
    f = mq.mq_mx4_gemm_bf16_workspace_bytes
    assert f(1, 4096, 4096) == f(2, 28672, 8192) == f(4, 4096, 4096) == f(3, 16384, 4096) == 0
    assert f(5, 4096, 4096) == 40 * 2048 + 32 * 512 and f(4, 28672, 8192) == 32 * 4096 + 64 * 512
    for M, N, K in ((0, 4, 32), (1, 0, 32), (1, 4, 33), (1 << 30, 4, 32)):
        assert mq.mq_mx4_gemm_bf16_workspace_bytes(M, N, K) == 0


def _m(rows=4, K=64, codes=FAKE, scales=FAKE * 2):
    return mq.MqMx4(codes, scales, rows, K)


@pytest.mark.parametrize("want,args", [
    (INVALID, (None, 0, 4, 64, 64, FAKE, FAKE)),
    (INVALID, (FAKE, 0, 4, 64, 64, None, FAKE)),
    (INVALID, (FAKE, 0, 4, 64, 64, FAKE, None)),
    (INVALID, (FAKE, 3, 4, 64, 64, FAKE, FAKE)),                  # dtype
    (INVALID, (FAKE, 0, 4, 48, 64, FAKE, FAKE)),                  # K
    (INVALID, (FAKE, 0, -1, 64, 64, FAKE, FAKE)),
    (INVALID, (FAKE, 0, 4, 64, 32, FAKE, FAKE)),                  # ld < K
    (MISALIGNED, (FAKE + 2, 0, 4, 64, 64, FAKE, FAKE)),
    (MISALIGNED, (FAKE, 0, 4, 64, 68, FAKE, FAKE)),               # 136-byte rows
    (MISALIGNED, (FAKE, 2, 4, 64, 66, FAKE, FAKE)),
    (MISALIGNED, (FAKE, 0, 4, 64, 64, FAKE + 8, FAKE)),
    (MISALIGNED, (FAKE, 0, 4, 64, 64, FAKE, FAKE + 4)),
    (0, (None, 0, 0, 64, 64, None, None)),                        # no rows: nothing to do
])
def test_quantize_refusals(want, args):
    assert mq.lib.mq_mx4_quantize(*args, None) == want


def test_from_nested_refusals():
    f = mq.lib.mq_mx4_from_nested
    w = mq.MqWeights(FAKE, FAKE, 64, 256, 128, 4)
    assert f(None, FAKE, FAKE, None) == INVALID
    assert f(ctypes.byref(w), None, FAKE, None) == INVALID
    assert f(ctypes.byref(w), FAKE, FAKE + 2, None) == MISALIGNED
    for bad in (mq.MqWeights(FAKE, FAKE, 64, 200, 128, 4), mq.MqWeights(FAKE, FAKE, 64, 256, 128, 9),
                mq.MqWeights(None, FAKE, 64, 256, 128, 4), mq.MqWeights(FAKE, FAKE, 0, 256, 128, 4)):
        assert f(ctypes.byref(bad), FAKE, FAKE, None) == INVALID


def test_dequantize_refusals():
    f = mq.lib.mq_mx4_dequantize
    ok = _m()
    assert f(None, FAKE, 0, 64, None) == INVALID
    assert f(ctypes.byref(ok), None, 0, 64, None) == INVALID
    assert f(ctypes.byref(ok), FAKE, 1, 64, None) == INVALID      # fp16 does not hold every value
    assert f(ctypes.byref(ok), FAKE, 0, 32, None) == INVALID
    assert f(ctypes.byref(ok), FAKE, 0, 65, None) == MISALIGNED
    assert f(ctypes.byref(ok), FAKE + 4, 2, 64, None) == MISALIGNED
    assert f(ctypes.byref(_m(codes=None)), FAKE, 0, 64, None) == INVALID
    assert f(ctypes.byref(_m(scales=FAKE + 1)), FAKE, 0, 64, None) == MISALIGNED
    assert f(ctypes.byref(_m(K=40)), FAKE, 0, 64, None) == INVALID
    assert f(ctypes.byref(_m(rows=0, codes=None, scales=None)), None, 0, 64, None) == 0


def test_gemm_refusals():
    f = mq.lib.mq_mx4_gemm
    call = lambda X, w, Y=FAKE, dt=0, ldy=8: f(ctypes.byref(X) if X else None, ctypes.byref(w) if w else None,
                                               Y, dt, ldy, None)
    x, w = _m(4), _m(8)
    assert call(None, w) == INVALID
    assert call(x, None) == INVALID
    assert call(x, _m(8, 96)) == INVALID                          # K differs
    assert call(x, _m(0)) == INVALID
    assert call(x, w, Y=None) == INVALID
    assert call(x, w, Y=FAKE + 2) == MISALIGNED
    assert call(x, w, dt=5) == INVALID
    assert call(x, w, ldy=7) == INVALID
    assert call(x, _m(8, codes=None)) == INVALID
    assert call(_m(4, codes=FAKE + 8), w) == MISALIGNED
    assert call(_m(0, codes=None, scales=None), w, Y=None) == 0   # no rows of X


def test_gemm_bf16_refusals():
    f = mq.lib.mq_mx4_gemm_bf16
    w = _m(8)
    need = mq.mq_mx4_gemm_bf16_workspace_bytes(40, 8, 64)
    call = lambda X=FAKE, M=40, ldx=64, w=w, Y=FAKE, dt=0, ldy=8, ws=FAKE, nb=need: \
        f(X, M, ldx, ctypes.byref(w) if w else None, Y, dt, ldy, ws, nb, None)
    assert call(X=None) == INVALID
    assert call(w=None) == INVALID
    assert call(M=-1) == INVALID
    assert call(M=1 << 40) == INVALID
    assert call(ldx=56) == INVALID
    assert call(ldx=68) == MISALIGNED
    assert call(X=FAKE + 2) == MISALIGNED
    assert call(ws=FAKE + 2) == MISALIGNED
    assert call(Y=None) == INVALID
    assert call(Y=FAKE + 4) == MISALIGNED
    assert call(dt=-1) == INVALID
    assert call(ldy=4) == INVALID
    assert call(ws=None) == WORKSPACE
    assert call(nb=need - 1) == WORKSPACE
    assert call(M=0, X=None, Y=None, ws=None) == 0


def test_binding_refuses_what_the_pointers_cannot_show():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        mq.mx4_quantize(x)
    with pytest.raises(ValueError, match="2-D"):
        mq.mx4_quantize(x[0])
    with pytest.raises(ValueError, match="GPU"):
        mq.Mx4Matrix(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)
    with pytest.raises(ValueError, match="GPU"):
        mq.Mx4Matrix.empty(4, 64, "cpu")
