"""What the bf16 product keeps of X: through an identity the product returns X
itself, so that each element shows its own error.

Bound: the slices leave less than 2^-22 of the largest value of each block of
32, whatever the number of rows and the output type.  Nothing is added to it: an
identity leaves one product an output, its slices are multiples of half the last
unit, 2^(e0 - 21), below 2^(e0 + 3), so that their fp32 sum is exact; then half
a step of the output type.  The rows are those that tell eight slices from
seven (tests/test_oracle_mx4_slices.py)."""
import numpy as np
import pytest

from tests.test_oracle_mx4_slices import block_max, telling_rows

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}          # half the smallest fp16


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _identity(K):
    import torch
    import nested_bit_weight_b200 as mq
    return mq.mx4_quantize(torch.eye(K, dtype=torch.bfloat16, device="cuda"))


def _dev(x):
    import torch
    return torch.from_numpy(x).cuda().bfloat16()


# cut inside the product (up to four rows), by a kernel of its own (four rows of
# large weights, five to sixteen rows), and for the product of CTA pairs
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 256), (2, 256), (3, 256), (4, 256), (4, 8448), (5, 256), (16, 256), (17, 256),
                                 (25, 288), (33, 256), (100, 256), (300, 544)])
def test_an_identity_returns_x(M, K, out):
    import nested_bit_weight_b200 as mq
    x = telling_rows(M, K, M + K)
    Y = mq.mx4_gemm_bf16(_dev(x), _identity(K), dtype=_dt(out)).double().cpu().numpy()
    X = x.astype(np.float64)
    left = 2.0 ** -22 * block_max(x)
    err = np.abs(Y - X)
    lim = left + EPS[out] * (np.abs(X) + left) + TINY[out]
    assert (err <= lim).all(), (int((err > lim).sum()), float((err / lim).max()))


def test_rows_do_not_depend_on_the_batch_or_the_output_type():
    # through an identity every form returns the same sums of slices
    import torch
    import nested_bit_weight_b200 as mq
    K = 256
    x, w = _dev(telling_rows(300, K, 9)), _identity(K)
    full = mq.mx4_gemm_bf16(x, w, dtype=torch.float32)
    for M in (1, 2, 4, 5, 16, 17, 24, 25, 32, 33, 100, 300):
        for dt in (torch.float32, torch.bfloat16, torch.float16):
            assert torch.equal(mq.mx4_gemm_bf16(x[:M], w, dtype=dt), full[:M].to(dt)), (M, dt)
    mq.mq_device_status()


def test_a_tile_of_more_than_24_rows():
    # 4096 features by 100 rows: 64 tiles of 25 rows instead of 80 of 20
    import torch
    import nested_bit_weight_b200 as mq
    K, N, M = 544, 4096, 100
    x = telling_rows(M, K, 4)
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    cols = torch.from_numpy(np.random.default_rng(1).integers(0, K, N)).cuda()
    w[torch.arange(N, device="cuda"), cols] = 1.0
    Y = mq.mx4_gemm_bf16(_dev(x), mq.mx4_quantize(w), dtype=torch.float32).double().cpu().numpy()
    sel = cols.cpu().numpy()
    X, left = x.astype(np.float64)[:, sel], (2.0 ** -22 * block_max(x))[:, sel]
    err = np.abs(Y - X)
    assert (err <= left + 2.0 ** -24 * (np.abs(X) + left)).all(), float((err / left).max())
    mq.mq_device_status()
