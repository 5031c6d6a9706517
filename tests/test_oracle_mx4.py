"""Pins of the MXFP4 oracle (oracle/mx4.py), from the definition alone."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mx4


def _nearest(x: Fraction):
    """Index of the grid point nearest to x >= 0 (ties to the even index)."""
    grid = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]
    best = min(abs(x - g) for g in grid)
    hits = [i for i, g in enumerate(grid) if abs(x - g) == best]
    return hits[0] if len(hits) == 1 else [i for i in hits if i % 2 == 0][0]


def test_codes_against_exact_rationals():
    rng = np.random.default_rng(7)
    v = rng.standard_normal((6, 64)) * np.exp2(rng.integers(-40, 40, (6, 1)))
    v[0, :32] = 0.0
    v[1, :16] = np.arange(16) / 4.0 * np.abs(v[1]).max()          # many ties
    codes, E = mx4.quantize(v)
    for r in range(6):
        for b in range(2):
            blk = [Fraction(float(x)) for x in v[r, 32 * b:32 * b + 32]]
            a = max(abs(x) for x in blk)
            if a == 0:
                assert E[r, b] == 0
                continue
            e = -127
            while Fraction(2) ** (e + 3) <= a:                     # floor(log2 a) = e + 2
                e += 1
            assert int(E[r, b]) == e + 127
            for j, x in enumerate(blk):
                want = _nearest(abs(x) / Fraction(2) ** e) + (8 if x < 0 else 0)
                got = int(codes[r, 32 * b + j])
                assert got == want or (x == 0 and got in (0, 8))


def test_worked_example():
    # largest 5: floor(log2 5) = 2, unit 1; the ties 0.25, 0.75, 2.5, 3.5, 5 go
    # to the even index (0, 2, 4, 6, 6)
    v = np.zeros((1, 32))
    v[0, :8] = [5.0, 0.25, 0.75, 2.5, 3.5, -1.25, -0.26, 1.75]
    codes, E = mx4.quantize(v)
    assert E[0, 0] == 127
    assert codes[0, :8].tolist() == [6, 0, 2, 4, 6, 8 + 2, 8 + 1, 4]
    assert mx4.round_trip(v)[0, :8].tolist() == [4.0, 0.0, 1.0, 2.0, 4.0, -1.0, -0.5, 2.0]


def test_top_of_the_range_and_the_smallest_scale():
    v = np.zeros((3, 32))
    v[0, 0] = 7.99                                                 # above 6: 6
    v[1, 0] = 2.0 ** -149                                          # floor(log2) - 2 < -127
    v[2, 0] = np.finfo(np.float32).max
    codes, E = mx4.quantize(v)
    assert (E[0, 0], codes[0, 0]) == (127, 7)
    assert (E[1, 0], codes[1, 0]) == (0, 0)
    assert (E[2, 0], codes[2, 0]) == (127 + 125, 7)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_block_with_a_non_finite_value_is_nan(bad):
    v = np.ones((2, 64))
    v[1, 40] = bad
    codes, E = mx4.quantize(v)
    assert E.tolist() == [[125, 125], [125, 255]] and not codes[1, 32:].any()
    rt = mx4.round_trip(v)
    assert np.isnan(rt[1, 32:]).all() and np.array_equal(rt[1, :32], v[1, :32])


def test_values_on_the_grid_are_kept():
    # numbers the format holds come back unchanged, also when the block's own
    # scale differs from the one they were made with
    rng = np.random.default_rng(3)
    c = rng.integers(0, 16, (20, 96)).astype(np.uint8)
    E = rng.integers(20, 230, (20, 3)).astype(np.uint8)
    v = mx4.values(c, E)
    assert np.array_equal(mx4.round_trip(v), v)


def test_storage_places():
    # one scale byte at a time lands where the layout formula says
    rows, K = 130, 288
    codes = np.zeros((rows, K), np.uint8)
    G = 3
    for n, j in ((0, 0), (31, 3), (32, 0), (127, 7), (128, 8), (129, 4)):
        E = np.zeros((rows, K // 32), np.uint8)
        E[n, j] = 77
        buf = mx4.pack(codes, E)[1]
        at = ((n // 128) * G + j // 4) * 512 + (n % 32) * 16 + ((n // 32) % 4) * 4 + j % 4
        assert buf.size == 2 * G * 512 and buf[at] == 77 and buf.sum() == 77
    codes[5, 6], codes[5, 7] = 3, 12
    assert mx4.pack(codes, np.zeros((rows, K // 32), np.uint8))[0][5, 3] == 3 | 12 << 4


def _mutants():
    def ties_away(u):
        return np.argmin(np.abs(u[..., None] - mx4.GRID) - 1e-9 * np.arange(8), axis=-1)
    def trunc(u):
        return np.searchsorted(mx4.GRID, u, side="right") - 1
    return {"ties away from zero": ties_away, "cut instead of rounded": trunc}


@pytest.mark.parametrize("name", list(_mutants()))
def test_planted_mistakes_differ_on_the_worked_example(name):
    u = np.array([5.0, 0.25, 0.75, 2.5, 3.5, 1.25, 0.26, 1.75])
    assert _mutants()[name](u).tolist() != [6, 0, 2, 4, 6, 2, 1, 4]
