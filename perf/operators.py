"""The microscaled 4-bit (MXFP4) operators as they are measured: cases, inputs,
plain forms in elementary torch operations, and the 64-bit definition.

Format: blocks of 32 consecutive columns share a scale 2^e, with
e = max(floor(log2 max|v|) - 2, -127); an element is v 2^-e rounded to
{0, .5, 1, 1.5, 2, 3, 4, 6} (nearest, ties to the even code, above 6 to 6).

Kinds of cases:
  quantize   dense rows -> MXFP4, returned as the bf16 values it stands for
  nested     an r-bit view of a nested parent -> MXFP4, returned the same way
  product4   Y = X4 . W4^T, X quantised within the call, W kept in MXFP4
  product16  Y = X . W4^T with X in bf16 as it is, W kept in MXFP4
"""
import math

import torch

own = False

GROUP = 128           # columns per scale of a nested parent
BLOCK = 32            # columns per scale of MXFP4

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token's activations before a 4-bit product: launch latency
        dict(name="quantize-token", kind="quantize", rows=1, K=4096, dtype="bf16"),
        # activations of a ragged prompt before a down projection
        dict(name="quantize-prompt", kind="quantize", rows=1021, K=14336, dtype="fp16"),
        # a long prompt's hidden states
        dict(name="quantize-long-prompt", kind="quantize", rows=8192, K=4096, dtype="bf16"),
        # a gate projection's float weights, laid out once
        dict(name="quantize-weights", kind="quantize", rows=14336, K=4096, dtype="fp32"),
        # a key projection's 2-bit model
        dict(name="nested-k", kind="nested", N=1024, K=4096, r=2, zeros=False),
        # a gate projection's 4-bit model with zero points
        dict(name="nested-gate", kind="nested", N=14336, K=4096, r=4, zeros=True),
        # sixteen sequences decoding together, an output projection
        dict(name="product4-batch", kind="product4", M=16, N=4096, K=4096, out="bf16"),
        # a ragged prompt, odd output features, a last block of columns inside a tile, fp32 outputs
        dict(name="product4-ragged", kind="product4", M=333, N=5001, K=4128, out="fp32"),
        # a long prompt through a gate projection: the matrix units' rate
        dict(name="product4-prompt", kind="product4", M=4096, N=14336, K=4096, out="bf16"),
        # one token through a key projection: latency
        dict(name="product16-token-k", kind="product16", M=1, N=1024, K=4096, out="bf16"),
        # one token through a gate projection: the weights' bytes
        dict(name="product16-token-gate", kind="product16", M=1, N=14336, K=4096, out="bf16"),
        # a batch of 100 sequences through a down projection, activations kept in 16 bits
        dict(name="product16-batch", kind="product16", M=100, N=4096, K=14336, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["quantize", "nested", "product4", "product16"])
    if kind == "quantize":
        K = BLOCK * _log_int(rng, 1, 896)                       # 32 .. 28672
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        rows = _log_int(rng, 1, max(1, min(32768, (14336 * 4096) // K)))
        return dict(kind=kind, rows=rows, K=K, dtype=dtype)
    if kind == "nested":
        K = GROUP * _log_int(rng, 1, 224)
        N = _log_int(rng, 1, max(1, min(28672, (14336 * 4096) // K)))
        return dict(kind=kind, N=N, K=K, r=rng.randint(1, 8), zeros=rng.random() < 0.5)
    K = BLOCK * _log_int(rng, 1, 896)
    N = _log_int(rng, 1, max(1, min(28672, (1 << 27) // K)))
    cap = 4096 if kind == "product4" else 256
    work = 4096 * 14336 * 4096 if kind == "product4" else 100 * 4096 * 14336
    M = _log_int(rng, 1, max(1, min(cap, work // (N * K))))
    return dict(kind=kind, M=M, N=N, K=K, out=rng.choice(["bf16", "fp16", "fp32"]))


# ------------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + salt)
    return g


def _activations(rows, K, dtype, seed):
    """Hidden states: N(0, 1), about one channel in 64 twenty times larger."""
    g = _gen(seed, 1)
    x = torch.randn(rows, K, generator=g, device="cuda")
    big = torch.rand(K, generator=g, device="cuda") < 1 / 64
    x.mul_(torch.where(big, 20.0, 1.0))
    return x.to(dtype)


def _weights(N, K, dtype, seed):
    """Weights: N(0, 0.02^2), one entry in a hundred ten times larger."""
    g = _gen(seed, 2)
    w = torch.randn(N, K, generator=g, device="cuda").mul_(0.02)
    w.mul_(torch.where(torch.rand(N, K, generator=g, device="cuda") < 0.01, 10.0, 1.0))
    return w.to(dtype)


def _parent(N, K, zeros, seed):
    """Codes, scales and zero points of a nested parent (codes 0..255)."""
    g = _gen(seed, 3)
    t = torch.randn(N, K, generator=g, device="cuda").mul_(32.0).add_(127.5)
    codes = t.round_().clamp_(0, 255).to(torch.uint8)
    G = K // GROUP
    scales = torch.rand(N, G, generator=g, device="cuda").mul_(1.8e-3).add_(2e-4)
    z = torch.randn(N, G, generator=g, device="cuda").mul_(12.0).add_(128.0) if zeros else None
    return codes, scales, z


def prepare(case, seed):
    kind, K = case["kind"], case["K"]
    if kind == "quantize":
        make = _weights if case["dtype"] == "fp32" else _activations
        return dict(kind=kind, X=make(case["rows"], K, _DT[case["dtype"]], seed))
    if kind == "nested":
        codes, scales, z = _parent(case["N"], K, case["zeros"], seed)
        state = dict(kind=kind, r=case["r"])
        if own:
            import nested_bit_weight_b200 as mq
            state["parent"] = mq.pack_parent(codes, scales, zeros=z)
        else:
            state.update(codes=codes, scales=scales.half(), zeros=None if z is None else z.half())
        return state
    W = _weights(case["N"], K, torch.bfloat16, seed)
    state = dict(kind=kind, X=_activations(case["M"], K, torch.bfloat16, seed), out=_DT[case["out"]])
    if own:
        import nested_bit_weight_b200 as mq
        state["W"] = mq.mx4_quantize(W)
    else:
        state["W"] = _mx4(W.float())                            # the values, kept in 32 bits
    return state


# -------------------------------------------------------------- plain forms

def _pow2(e, dtype):
    """2^e exactly, from the bits of its 64-bit form."""
    return ((e.long() + 1023) << 52).view(torch.float64).to(dtype)


def _mx4(v):
    """The values of v's MXFP4 form, in v's type (fp32 or fp64)."""
    R, K = v.shape
    b = v.view(R, K // BLOCK, BLOCK)
    amax = b.abs().amax(2, keepdim=True)
    _, ex = torch.frexp(amax)                                   # amax = m 2^ex, 0.5 <= m < 1
    e = torch.where(amax > 0, ex - 3, torch.full_like(ex, -127)).clamp_(min=-127)
    u = b * _pow2(-e, v.dtype)
    a = u.abs()
    c = (0.5 * (a > 0.25).to(v.dtype)).add_((a >= 0.75).to(v.dtype), alpha=0.5)
    c.add_((a > 1.25).to(v.dtype), alpha=0.5).add_((a >= 1.75).to(v.dtype), alpha=0.5)
    c.add_((a > 2.5).to(v.dtype)).add_((a >= 3.5).to(v.dtype)).add_((a > 5.0).to(v.dtype), alpha=2.0)
    return (torch.where(u < 0, -c, c) * _pow2(e, v.dtype)).view(R, K)


def _plain(s):
    kind = s["kind"]
    if kind == "quantize":
        return _mx4(s["X"].float()).bfloat16()
    if kind == "nested":
        r, codes = s["r"], s["codes"]
        # 64 bits: scale times level has more bits than 32-bit floats hold, and a border decides the code
        level = (codes >> (8 - r)).double().mul_(2.0 ** (8 - r)).add_(2.0 ** (7 - r))
        z = s["zeros"].double().repeat_interleave(GROUP, 1) if s["zeros"] is not None else 128.0
        w = level.sub_(z).mul_(s["scales"].double().repeat_interleave(GROUP, 1))
        return _mx4(w).bfloat16()
    X = s["X"].float()
    if kind == "product4":
        X = _mx4(X)
    return (X @ s["W"].t()).to(s["out"])


def _own(s):
    import nested_bit_weight_b200 as mq
    kind = s["kind"]
    if kind == "quantize":
        return mq.mx4_dequantize(mq.mx4_quantize(s["X"]))
    if kind == "nested":
        return mq.mx4_dequantize(mq.mx4_from_nested(s["parent"], s["r"]))
    if kind == "product4":
        return mq.mx4_gemm(mq.mx4_quantize(s["X"]), s["W"], dtype=s["out"])
    return mq.mx4_gemm_bf16(s["X"], s["W"], dtype=s["out"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------- definition

def _mx4_exact(v):
    """The same values from the definition: a grid step for each number."""
    R, K = v.shape
    b = v.double().reshape(-1, BLOCK)
    amax = b.abs().max(1).values
    lg = torch.floor(torch.log2(amax))
    lg = torch.where(torch.exp2(lg + 1) <= amax, lg + 1, lg)    # log2 may round across a power of two
    lg = torch.where(torch.exp2(lg) > amax, lg - 1, lg)
    e = torch.where(amax > 0, (lg - 2).clamp(min=-127.0), torch.full_like(lg, -127.0))
    unit = torch.exp2(e)[:, None]
    a = b.abs() / unit
    step = torch.where(a >= 4, 2.0, torch.where(a >= 2, 1.0, 0.5)).double()
    q = (torch.round(a / step) * step).clamp(max=6.0)           # round: halves to even
    return (torch.sign(b) * q * unit).view(R, K)


def exact(case, seed):
    kind, K = case["kind"], case["K"]
    if kind == "quantize":
        make = _weights if case["dtype"] == "fp32" else _activations
        return _mx4_exact(make(case["rows"], K, _DT[case["dtype"]], seed))
    if kind == "nested":
        codes, scales, z = _parent(case["N"], K, case["zeros"], seed)
        N, r = case["N"], case["r"]
        q = torch.div(codes.double(), 2 ** (8 - r), rounding_mode="floor")
        u = (q + 0.5) * 2 ** (8 - r)
        off = z.half().double() if z is not None else torch.full_like(scales, 128.0, dtype=torch.float64)
        u = u.view(N, -1, GROUP) - off[:, :, None]
        return _mx4_exact((u * scales.half().double()[:, :, None]).view(N, K))
    W = _mx4_exact(_weights(case["N"], K, torch.bfloat16, seed))
    X = _activations(case["M"], K, torch.bfloat16, seed)
    X = _mx4_exact(X) if kind == "product4" else X.double()
    return torch.einsum("mk,nk->mn", X, W)


# ----------------------------------------------------------- least of a pass

def work(case):
    kind, K = case["kind"], case["K"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    mx4 = lambda n: n // 2 + n // 32                            # codes and scales of n elements
    if kind == "quantize":
        n = case["rows"] * K
        # read, the MXFP4 form written and read again for its values, the values written
        return {"bytes": n * size[case["dtype"]] + 2 * mx4(n) + 2 * n, "flops": 4 * n}
    if kind == "nested":
        N = case["N"]
        n = N * K
        scales = 2 * n // GROUP * (2 if case["zeros"] else 1)
        return {"bytes": n * case["r"] // 8 + scales + 2 * mx4(n) + 2 * n, "flops": 6 * n}
    M, N = case["M"], case["N"]
    out = M * N * size[case["out"]]
    return {"bytes": 2 * M * K + mx4(N * K) + out, "flops": 2 * M * N * K}
