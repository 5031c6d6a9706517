"""A nested parent to MXFP4 where scales carry a sign: -0.0, which packing
accepts, and negative scales in a caller's own view, which the products take as
they are.  The stored bytes are the definition's (oracle/mx4.py), with and
without zero points, by the ordinary form and by the one for unusual zero
points alike."""
import numpy as np
import pytest

import workloads as wl
from oracle import mx4 as ox

pytestmark = pytest.mark.gpu

RS = [1, 2, 3, 4, 5, 8]
# no zero points, ordinary ones, ones of the out-of-line form
ZEROS = {"none": None, "ordinary": 121.5, "unusual": 3.14159}


def _parent(N, K, seed, s, z):
    import torch
    import nested_bit_weight_b200 as mq
    codes = np.random.default_rng(seed).integers(0, 256, (N, K)).astype(np.uint8)
    codes[1, :] = 128                                              # level minus 128 is positive, and least
    zeros = None if z is None else np.full((N, K // 128), z, np.float32)
    p = mq.pack_parent(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda(),
                       zeros=None if zeros is None else torch.from_numpy(zeros).cuda())
    return codes, p


def _values(codes, s, r, z):
    """The weights in fp64, exactly (11 bits times at most 33)."""
    level = (codes >> (8 - r)).astype(np.float64) * 2.0 ** (8 - r) + 2.0 ** (7 - r)
    off = 128.0 if z is None else float(np.float16(z))
    return (level - off) * np.repeat(s.astype(np.float16).astype(np.float64), 128, axis=1)


def _check(m, v):
    codes, E = ox.quantize(v)
    packed, scales = ox.pack(codes, E)
    assert np.array_equal(m.scales.cpu().numpy(), scales)
    assert np.array_equal(m.codes.cpu().numpy(), packed)


@pytest.mark.parametrize("z", list(ZEROS))
@pytest.mark.parametrize("r", RS)
def test_scales_of_minus_zero(r, z):
    import nested_bit_weight_b200 as mq
    N, K = 130, 384
    s = wl.gen_scales(N, K, r)
    s[::3, 0] = -0.0
    s[1::4, 2] = -0.0
    s[5, 1] = 0.0
    codes, p = _parent(N, K, r, s, ZEROS[z])
    _check(mq.mx4_from_nested(p, r), _values(codes, s, r, ZEROS[z]))


@pytest.mark.parametrize("z", list(ZEROS))
@pytest.mark.parametrize("r", RS)
def test_negative_scales_of_a_callers_view(r, z):
    import torch
    import nested_bit_weight_b200 as mq
    N, K = 40, 256
    s = wl.gen_scales(N, K, 50 + r)
    s[3, 1] = 0.0
    codes, p = _parent(N, K, 50 + r, s, ZEROS[z])
    p.scales16.view(torch.int16).bitwise_or_(-0x8000)              # the sign of every scale
    torch.cuda.synchronize()
    _check(mq.mx4_from_nested(p, r), _values(codes, -s, r, ZEROS[z]))


@pytest.mark.parametrize("M", [1, 6, 40, 300])
def test_products_with_scales_of_minus_zero(M):
    # zero weights give zeros beside the largest activations too: the products
    # equal those with +0.0 in the scales' place
    import torch
    import nested_bit_weight_b200 as mq
    N, K = 200, 384
    s = wl.gen_scales(N, K, 7)
    s[:, 0] = 0.0
    x = torch.from_numpy(np.random.default_rng(M).standard_normal((M, K)).astype(np.float32)).cuda()
    x[:, :128] *= 2.0 ** 100
    x = x.bfloat16()
    _, plus = _parent(N, K, 7, s, None)
    s[:, 0] = -0.0
    _, minus = _parent(N, K, 7, s, None)
    a, b = mq.mx4_from_nested(plus, 4), mq.mx4_from_nested(minus, 4)
    for dt in (torch.float32, torch.bfloat16):
        want, got = mq.mx4_gemm_bf16(x, a, dtype=dt), mq.mx4_gemm_bf16(x, b, dtype=dt)
        assert torch.isfinite(want).all() and torch.equal(got, want)
        want, got = mq.mx4_gemm(mq.mx4_quantize(x), a, dtype=dt), mq.mx4_gemm(mq.mx4_quantize(x), b, dtype=dt)
        assert torch.isfinite(want).all() and torch.equal(got, want)
