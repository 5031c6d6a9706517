"""MXFP4 (blocks of 32 columns, e2m1 elements, one power-of-two scale) by its
definition, in numpy fp64: what the GPU converters and products are checked
against.  Shares nothing with the library.

    e    = max(floor(log2 a) - 2, -127), a = max |v| of the block; E = e + 127
    code = nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} to |v| 2^-e, ties to the even
           index, plus 8 for a set sign bit
    a NaN or an infinity in the block: E = 255, codes 0, every value NaN
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def quantize(v: np.ndarray):
    """v [rows, K] (exact in fp64) -> (codes uint8 [rows, K], E uint8 [rows, K/32])."""
    v = np.asarray(v, np.float64)
    rows, K = v.shape
    b = v.reshape(rows, K // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    safe = np.where(bad[:, :, None], 0.0, b)
    a = np.abs(safe).max(axis=2)
    _, ex = np.frexp(a)                                  # a = m 2^ex, 0.5 <= m < 1
    e = np.where(a > 0, np.maximum(ex - 3, -127), -127).astype(np.int64)
    u = np.abs(np.ldexp(safe, -e[:, :, None]))
    # index of the nearest grid point: distances to both neighbours, the even one on a tie
    hi = np.clip(np.searchsorted(GRID, u, side="left"), 1, 7)
    dl, dh = u - GRID[hi - 1], GRID[hi] - u
    idx = np.where(dl < dh, hi - 1, np.where(dl > dh, hi, np.where(hi % 2 == 0, hi, hi - 1)))
    codes = (idx + 8 * np.signbit(safe)).astype(np.uint8)
    codes[bad] = 0
    E = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(rows, K), E


def values(codes: np.ndarray, E: np.ndarray) -> np.ndarray:
    """The fp64 values of codes [rows, K] under the scale bytes E [rows, K/32]."""
    s = np.where(E == 255, np.nan, np.ldexp(1.0, E.astype(np.int64) - 127))
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(s, BLOCK, axis=1)


def round_trip(v: np.ndarray) -> np.ndarray:
    return values(*quantize(v))


def pack(codes: np.ndarray, E: np.ndarray):
    """The two stored buffers: codes two a byte (even column low), scale bytes
    in 512-byte blocks of 128 rows x 128 columns, written entry by entry."""
    rows, K = codes.shape
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    G, T = (K + 127) // 128, (rows + 127) // 128
    buf = np.zeros((T, G, 512), np.uint8)
    n, j = np.meshgrid(np.arange(rows), np.arange(K // BLOCK), indexing="ij")
    buf[n // 128, j // 4, (n % 32) * 16 + (n % 128 // 32) * 4 + j % 4] = E
    return packed, buf.reshape(-1)


def product_bound(X: np.ndarray, W: np.ndarray, adds: int, out_eps: float, tiny: float = 0.0):
    """(Y, bound): the fp64 product X W^T and how far an fp32 sum of its terms,
    in any order of at most `adds` additions a term takes part in, each off by
    at most 2^-23 of its result (cut or rounded), may be from it, plus half a
    step of the output type (relative out_eps, at least tiny)."""
    Y = X @ W.T
    mag = np.abs(X) @ np.abs(W).T
    err = adds * 2.0 ** -23 * mag
    return Y, err + out_eps * (np.abs(Y) + err) + tiny


def slices(x: np.ndarray, count: int) -> list:
    """x [rows, K] (bf16 numbers) as the values of `count` MXFP4 matrices, a
    greedy sum: the first has the least unit 2^e0 with a <= 7 2^e0 in each
    block, the second a quarter of it, each later one an eighth of the one
    before (units of at least 2^-127); each is the nearest grid point to what
    the ones before leave."""
    rows, K = x.shape
    rest = np.asarray(x, np.float64).reshape(rows, K // BLOCK, BLOCK).copy()
    a = np.abs(rest).max(axis=2)
    m, ex = np.frexp(a)                                  # a = m 2^ex, 0.5 <= m < 1
    e = np.where(a > 0, ex - 3 + (m > 0.875), -127)      # 7 2^e0 = 0.875 2^(e0 + 3)
    out = []
    for j in range(count):
        unit = np.ldexp(1.0, np.maximum(e - (3 * j - 1 if j else 0), -127))[:, :, None]
        u = np.abs(rest) / unit
        hi = np.clip(np.searchsorted(GRID, u, side="left"), 1, 7)
        dl, dh = u - GRID[hi - 1], GRID[hi] - u
        idx = np.where(dl < dh, hi - 1, np.where(dl > dh, hi, np.where(hi % 2 == 0, hi, hi - 1)))
        q = np.copysign(GRID[idx], rest) * unit
        rest -= q
        out.append(q.reshape(rows, K))
    return out
