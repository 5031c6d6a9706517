"""Every form of the product of CTA pairs over several rounds of tiles, exact.

The operands are small multiples of powers of two, chosen so that every partial
sum is a multiple of 2^-6 below 2^18 (the slices of a bf16 row of sixteenths are
multiples of a sixteenth too), which fp32 holds whatever the order: the
outputs equal the fp64 product rounded once, element for element.  So a tile that
reads another's accumulator, a stage used twice or too early, scales of the wrong
rows or columns all show."""
import pytest

from tests.test_mx4_forms import CLUSTERS, FORMS, OUT, hooks, plan

pytestmark = pytest.mark.gpu

DT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def _mx4_rows(rows, K, seed):
    """A random MXFP4 matrix and its values: all codes, blocks scaled by 1/2 or 1."""
    import torch
    import nested_bit_weight_b200 as mq
    g = torch.Generator(device="cuda").manual_seed(seed)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    v = grid[torch.randint(0, 8, (rows, K), generator=g, device="cuda")]
    v = v * (1.0 - 2.0 * torch.randint(0, 2, (rows, K), generator=g, device="cuda"))
    v.view(rows, K // 32, 32)[:, :, 0] = 6.0                       # the block's scale is as drawn
    v *= torch.randint(1, 3, (rows, K // 32, 1), generator=g, device="cuda").expand(-1, -1, 32).reshape(rows, K) / 2
    m = mq.mx4_quantize(v)
    assert torch.equal(mq.mx4_dequantize(m, dtype=torch.float32), v)
    return m, v.double()


def _bf16_rows(rows, K, seed):
    """Multiples of 1/16 below 16 with eight significant bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randint(-255, 256, (rows, K), generator=g, device="cuda") / 16.0)
    return x.bfloat16(), x.double()


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("form,bn,rounds,M,N,K,wider", FORMS)
def test_every_form_is_exact_over_its_rounds(form, bn, rounds, M, N, K, wider, out):
    import torch
    import nested_bit_weight_b200 as mq
    dt = getattr(torch, DT[out])
    got, width, tiles = plan(hooks(), M, N, K, out, N + wider, form == 8)
    assert (got, width) == (form, bn) and -(-tiles // CLUSTERS) >= rounds
    w, W = _mx4_rows(N, K, 2)
    x, X = _bf16_rows(M, K, 1) if form == 8 else _mx4_rows(M, K, 1)
    ref = X @ W.T
    # multiples of 2^-6 whose magnitudes add up to less than 2^18: 24 bits
    assert float((X.abs() @ W.abs().T).max()) < 2.0 ** 18
    want = ref.float().to(dt)
    buf = torch.full((M + 1, N + wider), 7.0, dtype=dt, device="cuda")
    for _ in range(2):
        (mq.mx4_gemm_bf16 if form == 8 else mq.mx4_gemm)(x, w, Y=buf[:M, :N])
        bad = (buf[:M, :N] != want).nonzero()
        assert bad.numel() == 0, (bad.shape[0], bad[:4].tolist())
        assert (buf[M] == 7).all() and (buf[:M, N:] == 7).all()
        buf[:M, :N] = 0
    mq.mq_device_status()
