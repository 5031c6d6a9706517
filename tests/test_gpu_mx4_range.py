"""The largest scale bytes a matrix from elsewhere may hold: values below 2^128
come back exactly, larger ones as infinities with their sign."""
import numpy as np
import pytest

from oracle import mx4 as ox

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_dequantize_at_the_top_of_the_scales(dtype):
    import torch
    import nested_bit_weight_b200 as mq
    codes = np.tile(np.arange(16, dtype=np.uint8), (3, 6))          # every code, three blocks a row
    E = np.array([[252, 253, 254], [254, 252, 253], [0, 255, 254]], np.uint8)
    packed, scales = ox.pack(codes, E)
    m = mq.Mx4Matrix(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), 3, 96)
    v = ox.values(codes, E)
    want = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)
    assert np.isinf(want).any()
    got = mq.mx4_dequantize(m, dtype=getattr(torch, dtype)).double().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    assert (np.signbit(got) == np.signbit(v))[~np.isnan(v)].all()
