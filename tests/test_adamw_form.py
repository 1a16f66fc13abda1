"""What the header says of the 8-bit form of v (CPU, the tests' reference)."""

import numpy as np

import around_reference as ref

LEAST = 1.25 * 2.0 ** -32


def test_errors_of_the_kept_ratio():
    """An error is at most r/16, and below the least code that code, up to the
    FP32 product that gives r (2^-23 of it)."""
    rng = np.random.default_rng(3)
    r = 2.0 ** rng.uniform(-45, 0, 64 * 4000)
    r[::7] = np.ldexp(1 + (2 * rng.integers(0, 8, r[::7].size) + 1) / 16, -rng.integers(1, 33, r[::7].size))  # halfway
    r = r.astype(np.float32)
    r[::64] = 1
    codes, scales = ref.keep_v(r)
    off = np.abs(ref.kept_v(codes, scales).astype(np.float64) - r)
    least = r < LEAST
    assert least.any() and (codes[least] == 1).all() and (off[least] <= LEAST).all()
    assert (off[least] > r[least]).any()  # (far more than r/16)
    assert (off[~least] <= r[~least] / 16 * (1 + 2.0 ** -20)).all()
    assert (codes[r == 1] == 255).all()
