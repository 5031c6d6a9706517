"""bf16 rows as sums of MXFP4 rows: what eight leave, by the oracle's own greedy
sum, and that rows made to show it tell eight from seven and from six."""
import numpy as np
import pytest

from oracle import mx4


def telling_rows(M: int, K: int, seed: int) -> np.ndarray:
    """bf16 numbers (in fp32): in every block of 32 one channel a thousand times
    the size of the ordinary ones, and others spread over 2^-4 .. 2^-20 of it,
    all with eight random significant bits."""
    rng = np.random.default_rng(seed)
    x = np.exp2(-rng.integers(4, 21, (M, K)).astype(np.float64)) * 1024.0
    x[:, rng.random(K) < 0.3] = 1.0
    big = np.arange(0, K, 32) + rng.integers(0, 32, K // 32)
    x[:, big] = 1024.0
    x *= rng.integers(128, 256, (M, K)) / 256.0 * rng.choice([-1.0, 1.0], (M, K))
    return x.astype(np.float32)


def block_max(x):
    x = np.abs(np.asarray(x, np.float64))
    return x.reshape(x.shape[0], -1, 32).max(axis=2).repeat(32, axis=1)


def worst(x, count):
    """The largest rest of `count` slices, in units of its block's largest |x|."""
    left = np.abs(x.astype(np.float64) - sum(mx4.slices(x, count)))
    return float((left / block_max(x)).max())


@pytest.mark.parametrize("M,K,seed", [(3, 256, 1), (100, 256, 2), (1, 8448, 3)])
def test_what_slices_leave(M, K, seed):
    x = telling_rows(M, K, seed)
    assert worst(x, 8) < 2.0 ** -22
    # one slice fewer, and the cut once taken for 16-bit outputs, are told apart
    assert worst(x, 7) > 2.0 ** -22
    assert worst(x, 6) > 2.0 ** -18


def test_slices_of_the_ends_of_the_range():
    x = np.zeros((2, 64), np.float32)
    x[0, :3] = [2.0 ** 127 * 1.9921875, -2.0 ** 120, 2.0 ** 105]
    x[0, 32:35] = [7.0, 5.0, -0.4375]                              # the largest a unit takes; a tie; seven sixteenths
    x[1, :3] = [2.0 ** -120, 2.0 ** -126 * 1.5, 2.0 ** -128]       # units stop at 2^-127
    s = mx4.slices(x, 8)
    assert np.array_equal(sum(s), x.astype(np.float64))
    assert s[0][0, 32:34].tolist() == [6.0, 4.0]
