"""MXFP4 on a GPU: converters bit for bit against the 64-bit definition
(oracle/mx4.py), products within bounds derived from their arithmetic.

Bound of a product (oracle.mx4.product_bound): the products of two elements and
two powers of two are exact; a term takes part in at most 64 additions inside
an MMA, one per MMA of its tile (K / 64), and 15 more (the parts of a split K,
the eight slices of a bf16 row), each off by at most 2^-23 of a partial sum,
which is at most the sum of magnitudes; then half a step of the output type.
bf16 rows: S slices leave at most 2^(e0 - 3 (S - 1)) of an element, where the
block's largest value is above 3.5 * 2^e0: below 2^-22 of it with eight slices
(fp32 outputs, up to 16 rows), below 2^-16 with six (16-bit outputs)."""
import ctypes

import numpy as np
import pytest

import workloads as wl
from oracle import mx4 as ox

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}          # half the smallest fp16


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _mq():
    import nested_bit_weight_b200 as mq
    return mq


def _dev(a, dtype="fp32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(_dt(dtype))


def _host(t):
    return t.double().cpu().numpy()


def _acts(M, K, seed, dtype="bf16"):
    """Activations with outlier channels, as stored in `dtype`."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K))
    x[:, rng.random(K) < 1 / 64] *= 20.0
    return _dev(x, dtype)


def _check_mx4(m, v):
    """m's stored bytes are those of v (fp64) by the definition."""
    codes, E = ox.quantize(v)
    packed, scales = ox.pack(codes, E)
    assert np.array_equal(m.scales.cpu().numpy(), scales)
    assert np.array_equal(m.codes.cpu().numpy(), packed)


# ------------------------------------------------------------------ converters

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 4096), (2, 64), (3, 96), (127, 160), (128, 128), (129, 288),
                                    (1000, 1056)])
def test_quantize_bytes(rows, K, dtype):
    mq = _mq()
    x = _acts(rows, K, rows * 7 + K, dtype)
    _check_mx4(mq.mx4_quantize(x), _host(x))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_ties_zeros_and_the_ends_of_the_range(dtype):
    import torch
    mq = _mq()
    t = np.zeros((12, 64))
    q = np.arange(32) / 4.0                                        # 0 .. 7.75: every tie of the grid
    t[0, :32], t[0, 32:] = q, -q
    t[1, :32] = q * 2.0 ** -13
    t[2, 5] = -0.0
    fi = torch.finfo(_dt(dtype))
    t[3, 0], t[3, 1] = fi.max, -fi.max
    t[3, 40] = fi.tiny
    t[4, :32] = fi.smallest_normal * np.linspace(-1, 1, 32)        # subnormals of the type
    t[4, 40] = fi.smallest_normal * fi.eps                         # the smallest number
    t[5, :] = fi.max / 2
    t[6, :] = 1.0
    t[6, 3] = fi.max                                               # one giant beside ones
    x = _dev(t, dtype)
    if dtype == "fp32":                                            # next to the ties
        x[7, :32] = torch.nextafter(x[0, :32], torch.tensor(1e9, device="cuda"))
        x[8, :32] = torch.nextafter(x[0, :32], torch.tensor(-1e9, device="cuda"))
        x[9, :32] = torch.nextafter(torch.exp2(torch.arange(-16.0, 16.0, device="cuda")),
                                    torch.tensor(0.0, device="cuda"))
    _check_mx4(mq.mx4_quantize(x), _host(x))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_non_finite_blocks(dtype):
    import torch
    mq = _mq()
    x = _acts(5, 128, 3, dtype)
    x[0, 0], x[1, 63], x[2, 64], x[3, 127] = float("nan"), float("inf"), float("-inf"), float("nan")
    m = mq.mx4_quantize(x)
    _check_mx4(m, _host(x))
    y = mq.mx4_dequantize(m)
    assert torch.isnan(y).view(5, 4, 32).all(2).nonzero().tolist() == [[0, 0], [1, 1], [2, 2], [3, 3]]


def test_quantize_strided_rows_and_given_buffers():
    import torch
    mq = _mq()
    big = _acts(70, 512, 11)
    x = big[3:69:2, 64:64 + 224]                                   # row stride 1024, offset 128 bytes
    out = mq.Mx4Matrix.empty(33, 224, "cuda:0")
    out.codes.fill_(0xAB)
    out.scales.fill_(0xCD)
    assert mq.mx4_quantize(x, out=out) is out
    _check_mx4(out, _host(x))
    # one row may have any stride, and a transposed matrix is refused
    _check_mx4(mq.mx4_quantize(big[4:5, 8:40]), _host(big[4:5, 8:40]))
    with pytest.raises(ValueError, match="contiguous rows"):
        mq.mx4_quantize(big.t())
    with pytest.raises(ValueError, match="overlap"):
        mq.mx4_quantize(big[:1].expand(4, 512))
    with pytest.raises(mq.MQError, match="MISALIGNED"):
        mq.mx4_quantize(big[:, 4:36])
    with pytest.raises(ValueError, match="multiple of 32"):
        mq.mx4_quantize(big[:, :40])
    with pytest.raises(ValueError, match="expected"):
        mq.mx4_quantize(x, out=mq.Mx4Matrix.empty(33, 256, "cuda:0"))
    with pytest.raises(ValueError, match="dtype"):
        mq.mx4_quantize(torch.zeros(2, 32, dtype=torch.float64, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (6, 96), (131, 416)])
def test_dequantize_every_code_and_scale(rows, K, dtype):
    import torch
    mq = _mq()
    rng = np.random.default_rng(rows)
    codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    E = rng.integers(0, 253, (rows, K // 32)).astype(np.uint8)
    E[0, 0] = 0
    E[-1, -1] = 255
    packed, scales = ox.pack(codes, E)
    m = mq.Mx4Matrix(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), rows, K)
    want = ox.values(codes, E)
    assert np.array_equal(_host(mq.mx4_dequantize(m, dtype=_dt(dtype))), want, equal_nan=True)
    # into a wider buffer: columns beyond K stay as they were
    buf = torch.full((rows, K + 64), 7.0, dtype=_dt(dtype), device="cuda")
    mq.mx4_dequantize(m, out=buf[:, 32:32 + K])
    assert np.array_equal(_host(buf[:, 32:32 + K]), want, equal_nan=True)
    assert (buf[:, :32] == 7).all() and (buf[:, 32 + K:] == 7).all()


def _nested(N, K, seed, zeros=None):
    import torch
    mq = _mq()
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (N, K)).astype(np.uint8)
    codes[0, :128] = 128
    s = wl.gen_scales(N, K, seed, zero_groups=1 if N > 1 else 0)
    p = mq.pack_parent(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda(),
                       zeros=None if zeros is None else torch.from_numpy(zeros).cuda())
    return codes, s, p


def _nested_values(codes, s, r, zeros=None):
    """W_r in fp64 (exact: 11 bits times at most 33)."""
    K = codes.shape[1]
    level = (codes >> (8 - r)).astype(np.float64) * 2.0 ** (8 - r) + 2.0 ** (7 - r)
    z = 128.0 if zeros is None else np.repeat(zeros.astype(np.float16).astype(np.float64), 128, axis=1)
    return (level - z) * np.repeat(s.astype(np.float16).astype(np.float64), 128, axis=1)[:, :K]


@pytest.mark.parametrize("r", range(1, 9))
@pytest.mark.parametrize("N,K", [(1, 128), (130, 384)])
def test_from_nested_bytes(N, K, r):
    codes, s, p = _nested(N, K, 10 * r + N)
    _check_mx4(_mq().mx4_from_nested(p, r), _nested_values(codes, s, r))


@pytest.mark.parametrize("r", [1, 3, 4, 8])
def test_from_nested_zero_points_of_every_size(r):
    # ordinary ones, ones at the borders of the 32-bit form, and ones whose
    # difference from a level needs more bits than fp32 has
    N, K = 40, 512
    rng = np.random.default_rng(r)
    z = rng.normal(128, 12, (N, K // 128)).astype(np.float32)
    z[:8, 0] = [32.0, 31.98, 4096.0, 4094.0, 0.0, -0.0, 1e-7, 6e-8]
    z[8:16, 1] = [0.1, -0.3, 3.14159, 17.77, -130.1, 65504.0, -65504.0, 20000.0]
    z[16:24, 2] = [127.5, 64.0, 32.03, 2047.0, 1e-3, 0.5, 255.9, 4100.0]
    codes, s, p = _nested(N, K, 77 + r, z)
    _check_mx4(_mq().mx4_from_nested(p, r), _nested_values(codes, s, r, z))


# -------------------------------------------------------------------- products

def _close(Y, X, W, K, out, extra=0.0):
    ref, bound = ox.product_bound(X, W, 64 + K // 64 + 1 + 15, EPS[out], TINY[out])
    err = np.abs(_host(Y) - ref)
    bad = err > bound + extra
    assert not bad.any(), (int(bad.sum()), float((err / (bound + extra + 1e-300)).max()))


def _rest(X, W, out="fp32"):
    """What the slices may leave: a share of each block's largest |x|."""
    a = np.abs(X).reshape(X.shape[0], -1, 32).max(2).repeat(32, axis=1)
    return (2.0 ** -22 if out == "fp32" or X.shape[0] <= 16 else 2.0 ** -16) * (a @ np.abs(W).T)


SHAPES = [(1, 1, 32), (1, 128, 64), (1, 1024, 4096), (2, 130, 96), (3, 300, 4128), (5, 4096, 2048), (8, 129, 1056),
          (16, 256, 14336), (17, 1000, 288), (33, 640, 512), (64, 128, 256), (65, 200, 544), (128, 384, 1024),
          (129, 128, 4096), (255, 257, 800), (300, 1280, 2080), (1000, 700, 160), (25, 260, 288), (31, 264, 96),
          (130, 5000, 512), (200, 5001, 512), (500, 640, 1312), (385, 321, 64), (300, 1, 64), (300, 300, 32),
          (2, 4096, 4096), (2, 5, 32), (3, 2000, 4096), (4, 1000, 14336), (4, 17000, 4096), (24, 7, 32), (129, 8, 4096), (12, 20000, 160)]


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K, out):
    mq = _mq()
    x, w = _acts(M, K, M + N + K), _dev(np.random.default_rng(N).standard_normal((N, K)) * 0.02, "bf16")
    W4, X4 = mq.mx4_quantize(w), mq.mx4_quantize(x)
    X, Wv = _host(x), ox.round_trip(_host(w))
    _close(mq.mx4_gemm(X4, W4, dtype=_dt(out)), ox.round_trip(X), Wv, K, out)
    _close(mq.mx4_gemm_bf16(x, W4, dtype=_dt(out)), X, Wv, K, out, _rest(X, Wv, out))
    mq.mq_device_status()


@pytest.mark.parametrize("M", [1, 4, 9, 40, 300])
def test_one_hot_rows_return_columns(M):
    # operand order, scale bytes and the K order of both operands: exact
    import torch
    mq = _mq()
    N, K = 200, 416
    rng = np.random.default_rng(M)
    W = ox.values(rng.integers(0, 16, (N, K)).astype(np.uint8), rng.integers(120, 130, (N, K // 32)).astype(np.uint8))
    w4 = mq.mx4_quantize(_dev(W))
    ks = rng.integers(0, K, M)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    scale = np.exp2(rng.integers(-3, 4, M))
    x[torch.arange(M), torch.from_numpy(ks)] = torch.from_numpy(scale).to(torch.bfloat16).cuda()
    want = (W[:, ks] * scale).T
    assert np.array_equal(_host(mq.mx4_gemm(mq.mx4_quantize(x), w4, dtype=torch.float32)), want)
    assert np.array_equal(_host(mq.mx4_gemm_bf16(x, w4, dtype=torch.float32)), want)


@pytest.mark.parametrize("M", [1, 7, 50])
def test_bf16_rows_of_any_size_of_numbers(M):
    # tiny, huge and mixed magnitudes, an all-zero block, subnormal bf16
    mq = _mq()
    N, K = 140, 288
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-12, 12, (M, K)))
    x[:, :32] *= 2.0 ** -100
    x[:, 32:64] *= 2.0 ** 60
    x[:, 64:96] = 0.0
    x[:, 96:128] = rng.integers(-3, 4, (M, 32)) * 2.0 ** -133
    xd = _dev(x, "bf16")
    X = _host(xd)
    w = rng.standard_normal((N, K))
    w[:, 32:64] *= 2.0 ** -60
    w4 = mq.mx4_quantize(_dev(w))
    Wv = ox.round_trip(_host(_dev(w)))
    _close(mq.mx4_gemm_bf16(xd, w4, dtype=_dt("fp32")), X, Wv, K, "fp32", _rest(X, Wv) + 2.0 ** -120)


@pytest.mark.parametrize("M,N", [(1, 130), (6, 130), (40, 1280), (300, 300)])
def test_non_finite_values_stay_in_their_row_and_feature(M, N):
    import torch
    mq = _mq()
    K = 512
    x, w = _acts(M, K, 5), _acts(N, K, 6)
    r = M // 2
    clean4 = mq.mx4_gemm(mq.mx4_quantize(x), mq.mx4_quantize(w))
    clean16 = mq.mx4_gemm_bf16(x, mq.mx4_quantize(w))
    for bad in (float("nan"), float("inf")):
        xb, wb = x.clone(), w.clone()
        xb[r, 77] = bad
        wb[N - 1, 300] = bad
        w4 = mq.mx4_quantize(wb)
        for Y, clean in ((mq.mx4_gemm(mq.mx4_quantize(xb), w4), clean4), (mq.mx4_gemm_bf16(xb, w4), clean16)):
            nan = torch.isnan(Y)
            assert nan[r].all() and nan[:, N - 1].all()
            nan[r] = False
            nan[:, N - 1] = False
            assert not nan.any()
            keep = torch.ones_like(nan)
            keep[r] = False
            keep[:, N - 1] = False
            assert torch.equal(Y[keep], clean[keep])


@pytest.mark.parametrize("M,N,ldy", [(1, 130, 131), (3, 129, 200), (70, 128, 136), (300, 256, 257), (300, 250, 512)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_strided_outputs_and_inputs(M, N, ldy, out):
    import torch
    mq = _mq()
    K = 320
    xb = _acts(M, K + 96, 9)
    x = xb[:, 64:64 + K]
    w4 = mq.mx4_quantize(_acts(N, K, 10))
    X4 = mq.mx4_quantize(x)
    for fn, a in ((mq.mx4_gemm, X4), (mq.mx4_gemm_bf16, x)):
        want = fn(a, w4, dtype=_dt(out)) if fn is mq.mx4_gemm else fn(a.contiguous(), w4, dtype=_dt(out))
        buf = torch.full((M + 1, ldy), 5.0, dtype=_dt(out), device="cuda")
        assert fn(a, w4, Y=buf[:M, :N]) .data_ptr() == buf.data_ptr()
        assert torch.equal(buf[:M, :N], want)
        assert (buf[M] == 5).all() and (buf[:M, N:] == 5).all()


def test_binding_refusals_on_device():
    import torch
    mq = _mq()
    x, w4 = _acts(4, 64, 1), mq.mx4_quantize(_acts(8, 64, 2))
    with pytest.raises(ValueError, match="bfloat16"):
        mq.mx4_gemm_bf16(x.float(), w4)
    with pytest.raises(ValueError, match="expected"):
        mq.mx4_gemm_bf16(x[:, :32], w4)
    with pytest.raises(mq.MQError, match="differ in K"):
        mq.mx4_gemm(mq.mx4_quantize(x[:, :32]), w4)
    with pytest.raises(ValueError, match="expected"):
        mq.mx4_gemm(mq.mx4_quantize(x), w4, Y=torch.empty(4, 9, device="cuda"))
    with pytest.raises(ValueError, match="dtype"):
        mq.mx4_gemm(mq.mx4_quantize(x), w4, dtype=torch.float64)
    with pytest.raises(ValueError, match="differs in dtype"):
        mq.mx4_gemm(mq.mx4_quantize(x), w4, Y=torch.empty(4, 8, device="cuda"), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiple of 32"):
        mq.Mx4Matrix.empty(4, 40, "cuda")
    # the default stream by its handle, and an event's stream as an object
    want = mq.mx4_gemm_bf16(x, w4)
    torch.cuda.synchronize()
    assert torch.equal(mq.mx4_gemm_bf16(x, w4, stream=0), want)
    assert torch.equal(mq.mx4_gemm_bf16(x, w4, stream=torch.cuda.default_stream()), want)


def test_no_rows():
    import torch
    mq = _mq()
    w4 = mq.mx4_quantize(_acts(8, 64, 2))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    X4 = mq.mx4_quantize(x)
    assert X4.rows == 0 and mq.mx4_dequantize(X4).shape == (0, 64)
    assert mq.mx4_gemm(X4, w4).shape == (0, 8)
    assert mq.mx4_gemm_bf16(x, w4).shape == (0, 8)


@pytest.mark.parametrize("M", [1, 8, 24, 200])
def test_repeated_calls_are_bit_equal(M):
    import torch
    mq = _mq()
    x, w4 = _acts(M, 4096, 1), mq.mx4_quantize(_acts(1000, 4096, 2))
    X4 = mq.mx4_quantize(x)
    a, b = mq.mx4_gemm(X4, w4, dtype=torch.float32), mq.mx4_gemm_bf16(x, w4, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(mq.mx4_gemm(X4, w4, dtype=torch.float32), a)
        assert torch.equal(mq.mx4_gemm_bf16(x, w4, dtype=torch.float32), b)


# ------------------------------------------------- streams, graphs, two at once

@pytest.mark.parametrize("M", [1, 12, 300])
def test_two_streams_at_once_and_explicit_streams(M):
    import torch
    mq = _mq()
    w4 = [mq.mx4_quantize(_acts(2000, 4096, s)) for s in (1, 2)]
    xs = [_acts(M, 4096, 10 + s) for s in (1, 2)]
    want = [(mq.mx4_gemm(mq.mx4_quantize(x), w), mq.mx4_gemm_bf16(x, w)) for x, w in zip(xs, w4)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for rep in range(6):
        for i in (0, 1):
            if rep % 2:                                            # named by the argument, also as a raw handle
                s = st[i] if rep % 4 == 1 else st[i].cuda_stream
                got.append((i, mq.mx4_gemm(mq.mx4_quantize(xs[i], stream=s), w4[i], stream=s),
                            mq.mx4_gemm_bf16(xs[i], w4[i], stream=s)))
            else:
                with torch.cuda.stream(st[i]):
                    got.append((i, mq.mx4_gemm(mq.mx4_quantize(xs[i]), w4[i]), mq.mx4_gemm_bf16(xs[i], w4[i])))
    torch.cuda.synchronize()
    mq.mq_device_status()
    for i, a, b in got:
        assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])


def test_two_host_threads_at_once():
    import threading
    import torch
    mq = _mq()
    w4 = mq.mx4_quantize(_acts(1500, 2048, 1))
    xs = [_acts(M, 2048, M) for M in (3, 150)]
    want = [(mq.mx4_gemm(mq.mx4_quantize(x), w4), mq.mx4_gemm_bf16(x, w4)) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(40):
                    y = mq.mx4_gemm(mq.mx4_quantize(xs[i]), w4), mq.mx4_gemm_bf16(xs[i], w4)
            st.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(y, want[i])):
                bad.append(i)
        except Exception as e:                                     # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i % 2,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    mq.mq_device_status()
    assert not bad, bad


@pytest.mark.parametrize("M", [1, 20, 200])
def test_captured_graphs_replayed_with_new_inputs_and_side_by_side(M):
    import torch
    mq = _mq()
    K, N = 1056, 700
    w4 = mq.mx4_quantize(_acts(N, K, 3))
    xin = [_acts(M, K, 20 + i) for i in (0, 1)]
    mq.mx4_gemm_bf16(xin[0], w4)                                   # first use outside a capture
    graphs, outs = [], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            X4 = mq.mx4_quantize(xin[i])
            outs.append((mq.mx4_dequantize(X4), mq.mx4_gemm(X4, w4), mq.mx4_gemm_bf16(xin[i], w4)))
        graphs.append(g)
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        new = [_acts(M, K, 100 * rep + i) for i in (0, 1)]
        for i in (0, 1):
            xin[i].copy_(new[i])
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(st[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        mq.mq_device_status()
        for i in (0, 1):
            X4 = mq.mx4_quantize(new[i])
            want = (mq.mx4_dequantize(X4), mq.mx4_gemm(X4, w4), mq.mx4_gemm_bf16(new[i], w4))
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want))


def test_first_calls_of_a_process_inside_a_capture():
    # nothing is set up lazily that a capture does not allow
    import os
    import subprocess
    import sys
    code = """
import torch
import nested_bit_weight_b200 as mq
torch.manual_seed(1)
x, xb = (torch.randn(m, 512, device='cuda').bfloat16() for m in (1, 300))
w = torch.randn(384, 512, device='cuda').bfloat16()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    w4 = mq.mx4_quantize(w)
    out = [mq.mx4_gemm_bf16(x, w4), mq.mx4_gemm(mq.mx4_quantize(x), w4), mq.mx4_gemm_bf16(xb, w4),
           mq.mx4_gemm(mq.mx4_quantize(xb), w4), mq.mx4_dequantize(w4)]
g.replay()
torch.cuda.synchronize()
w4 = mq.mx4_quantize(w)
want = [mq.mx4_gemm_bf16(x, w4), mq.mx4_gemm(mq.mx4_quantize(x), w4), mq.mx4_gemm_bf16(xb, w4),
        mq.mx4_gemm(mq.mx4_quantize(xb), w4), mq.mx4_dequantize(w4)]
assert all(torch.equal(a, b) for a, b in zip(out, want))
mq.mq_device_status()
print('captured first')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert "captured first" in r.stdout, r.stdout + r.stderr


def test_beside_and_between_the_nested_products():
    # one stream: nested and MXFP4 products in turn, each launched while the one
    # before still runs; two streams: both at once
    import torch
    mq = _mq()
    N, K = 1024, 4096
    codes, s, p = _nested(N, K, 3)
    w4 = mq.mx4_from_nested(p, 4)
    xs = {M: _acts(M, K, M) for M in (1, 16, 200)}
    want = {}
    for M, x in xs.items():
        want[M] = [mq.gemm(x, p, 2), mq.mx4_gemm_bf16(x, w4), mq.gemm(x, p, 4), mq.mx4_gemm(mq.mx4_quantize(x), w4)]
        torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for M, x in xs.items():
            got.append((M, [mq.gemm(x, p, 2), mq.mx4_gemm_bf16(x, w4), mq.gemm(x, p, 4),
                            mq.mx4_gemm(mq.mx4_quantize(x), w4)]))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    pair = []
    for _ in range(10):
        for M, x in xs.items():
            with torch.cuda.stream(a):
                y = mq.gemm(x, p, 2)
            with torch.cuda.stream(b):
                pair.append((M, y, mq.mx4_gemm_bf16(x, w4), mq.mx4_gemm(mq.mx4_quantize(x), w4)))
    torch.cuda.synchronize()
    mq.mq_device_status()
    for M, ys in got:
        assert all(torch.equal(u, v) for u, v in zip(ys, want[M]))
    for M, y, y16, y4 in pair:
        assert torch.equal(y, want[M][0]) and torch.equal(y16, want[M][1]) and torch.equal(y4, want[M][3])


def test_weights_quantized_right_before_the_product():
    # weights written by the call before: nothing of them may be read early
    import torch
    mq = _mq()
    x = _acts(1, 4096, 4)
    ws = [_acts(2048, 4096, 30 + i) for i in range(4)]
    out = mq.Mx4Matrix.empty(2048, 4096, "cuda:0")
    want = [mq.mx4_gemm_bf16(x, mq.mx4_quantize(w), dtype=torch.float32) for w in ws]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for w in ws:
            mq.mx4_quantize(w, out=out)
            got.append(mq.mx4_gemm_bf16(x, out, dtype=torch.float32))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 4])


# ------------------------------------------------------------ beyond 32 bits

def test_offsets_beyond_32_bits():
    import torch
    mq = _mq()
    rows, K = 66000, 65536                                         # 4.3e9 elements
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    tail = _acts(200, K, 8)
    x[-200:] = tail
    m = mq.mx4_quantize(x)
    want = mq.mx4_quantize(tail)
    assert torch.equal(m.codes[-200:], want.codes) and not m.codes[:-200].any()
    y = mq.mx4_dequantize(m)
    assert torch.equal(y[-200:], mq.mx4_dequantize(want)) and not y[:-200].any()
    del x, y
    # as weights (codes beyond 2^31 bytes) and as X with outputs beyond 2^31
    a = _acts(3, K, 9)
    assert torch.equal(mq.mx4_gemm_bf16(a, m)[:, -200:], mq.mx4_gemm_bf16(a, want))
    del m
    M, N, K2 = 70000, 32768, 64
    x, w4 = _acts(M, K2, 12), mq.mx4_quantize(_acts(N, K2, 13))
    Y = mq.mx4_gemm(mq.mx4_quantize(x), w4)
    for lo in (0, 65400, M - 300):
        assert torch.equal(Y[lo:lo + 300], mq.mx4_gemm(mq.mx4_quantize(x[lo:lo + 300]), w4))


# --------------------------------------------------------------- used together

def test_a_nested_parent_served_in_both_ways():
    """A nested parent's 4-bit model as MXFP4: a prompt through the 4-bit
    product, a token through the bf16 one, the same token through mq_gemm.
    The products agree with the dense values of the MXFP4 weights; mq_gemm of
    the parent differs by what the format rounds, at most 2^-2 of an element
    (a 2-bit significand: half a step is 1/4 at most below the top, where
    numbers above 6 lose a quarter)."""
    import torch
    mq = _mq()
    N, K = 1024, 512
    codes, s, _ = wl.gen_weights(N, K, seed=5)
    p = mq.pack_parent(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda())
    w4 = mq.mx4_from_nested(p, 4)
    W = _nested_values(codes, s, 4)
    Wv = ox.round_trip(W)
    assert np.array_equal(_host(mq.mx4_dequantize(w4)), Wv)
    prompt, token = _acts(77, K, 1), _acts(1, K, 2)
    _close(mq.mx4_gemm(mq.mx4_quantize(prompt), w4), ox.round_trip(_host(prompt)), Wv, K, "bf16")
    X = _host(token)
    y16 = mq.mx4_gemm_bf16(token, w4)
    _close(y16, X, Wv, K, "bf16", _rest(X, Wv))
    yn = mq.gemm(token, p, 4)
    a = np.abs(W).reshape(N, -1, 32).max(2).repeat(32, axis=1)
    # nearest grid point: off by at most a quarter of the number, or 2^-4 of the block's largest
    lim = np.abs(X) @ np.maximum(0.25 * np.abs(W), a / 8).T
    tol = 8e-3 * np.abs(X @ W.T) + 1e-3 * np.sqrt(np.mean((X @ W.T) ** 2))
    assert (np.abs(_host(y16) - _host(yn)) <= lim + tol + 2.0 ** -7 * np.abs(X @ Wv.T)).all()
    mq.mq_device_status()


# ------------------------------------------------------------ a wait that ends

def test_a_lost_load_ends_with_a_status():
    """Test-hook build: one CTA drops one load; its waits give up after 5 ms,
    the launch ends, the status says so once, and the next call is exact."""
    import torch
    from tests.test_gpu_timeout import MQ_ERR_TIMEOUT, _hooks_lib
    mq = _mq()
    L = _hooks_lib()
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    X4 = ctypes.POINTER(mq.MqMx4)
    L.mq_mx4_gemm.restype = I
    L.mq_mx4_gemm.argtypes = [X4, X4, P, I, I64, P]
    L.mq_test_drop_mx4_loads.argtypes = [I]
    for M, N, K in ((4, 300, 2048), (300, 1024, 1024)):
        x4, w4 = mq.mx4_quantize(_acts(M, K, 1)), mq.mx4_quantize(_acts(N, K, 2))
        want = mq.mx4_gemm(x4, w4)
        Y = torch.empty_like(want)
        torch.cuda.synchronize()
        args = (ctypes.byref(x4.struct), ctypes.byref(w4.struct), Y.data_ptr(), 0, N, None)
        assert L.mq_device_status() == 0
        assert L.mq_test_drop_mx4_loads(1) == 0
        assert L.mq_mx4_gemm(*args) == 0
        assert L.mq_device_status() == MQ_ERR_TIMEOUT
        assert L.mq_device_status() == 0
        Y.fill_(0)
        assert L.mq_mx4_gemm(*args) == 0 and L.mq_device_status() == 0
        assert torch.equal(Y, want)
