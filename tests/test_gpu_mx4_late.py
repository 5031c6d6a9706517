"""MXFP4 products whose K is split over the CTAs of a cluster, when a wait for
another CTA's parts runs out: a test-hook build (waits of 5 ms) makes CTAs drop
their loads, or send their parts only after the others have given up.  The
launch ends with a status, nothing is sent to a CTA that has ended, and the next
call on the same buffers is exact."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _lib():
    import nested_bit_weight_b200 as mq
    from tests.test_gpu_timeout import _hooks_lib
    L = _hooks_lib()
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    X4 = ctypes.POINTER(mq.MqMx4)
    L.mq_mx4_gemm.restype = L.mq_mx4_gemm_bf16.restype = I
    L.mq_mx4_gemm.argtypes = [X4, X4, P, I, I64, P]
    L.mq_mx4_gemm_bf16.argtypes = [P, I64, I64, X4, P, I, I64, P, SZ, P]
    L.mq_test_drop_mx4_loads.argtypes = L.mq_test_late_mx4_parts.argtypes = [I]
    return mq, L


def _dev(rows, K, seed):
    import torch
    x = np.random.default_rng(seed).standard_normal((rows, K)).astype(np.float32)
    return torch.from_numpy(x).cuda().bfloat16()


# K = 8192: 32 stages, eight CTAs a cluster; 2048: two.  With four rows or fewer
# only the first CTA of a cluster owns columns, with 100 all of them do.
@pytest.mark.parametrize("fault", ["late", "drop", "drop three"])
@pytest.mark.parametrize("kind,M,N,K", [("bf16", 1, 128, 8192), ("bf16", 2, 300, 2048), ("mx4", 4, 130, 8192),
                                        ("mx4", 16, 256, 8192), ("mx4", 100, 300, 8192)])
def test_parts_that_do_not_come_in_time(kind, M, N, K, fault):
    import torch
    from tests.test_gpu_timeout import MQ_ERR_TIMEOUT
    mq, L = _lib()
    x, w4 = _dev(M, K, 1), mq.mx4_quantize(_dev(N, K, 2))
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    if kind == "mx4":
        x4 = mq.mx4_quantize(x)
        want = mq.mx4_gemm(x4, w4)
        call = lambda: L.mq_mx4_gemm(ctypes.byref(x4.struct), ctypes.byref(w4.struct), Y.data_ptr(), 0, N, None)
    else:
        want = mq.mx4_gemm_bf16(x, w4)
        call = lambda: L.mq_mx4_gemm_bf16(x.data_ptr(), M, K, ctypes.byref(w4.struct), Y.data_ptr(), 0, N, None, 0, None)
    torch.cuda.synchronize()
    assert L.mq_device_status() == 0
    arm, on, off = (L.mq_test_late_mx4_parts, 1, 0) if fault == "late" else \
        (L.mq_test_drop_mx4_loads, 3 if fault == "drop three" else 1, 0)
    try:
        assert arm(on) == 0
        assert call() == 0
        assert L.mq_device_status() == MQ_ERR_TIMEOUT
    finally:
        assert arm(off) == 0
    assert L.mq_device_status() == 0                               # reported once
    for _ in range(2):
        Y.fill_(0)
        assert call() == 0 and L.mq_device_status() == 0
        assert torch.equal(Y, want)
