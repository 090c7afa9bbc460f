"""The oracle's bf16 rounding on values that are not finite, on the CPU."""

import numpy as np

import oracle


def test_infinities_stay_and_overflow_reaches_them():
    inf = np.inf
    top = 2.0**128 - 2.0**120  # the largest bf16
    half = 2.0**128 - 2.0**119  # halfway to the next power of two
    v = np.array([inf, -inf, top, np.nextafter(half, 0.0), half, -half, 1e300])
    assert np.array_equal(oracle.bf16_round(v), [inf, -inf, top, top, inf, -inf, inf])
    assert np.isnan(oracle.bf16_round(np.array([np.nan]))).all()


def test_norm_of_a_row_whose_residual_is_infinite():
    """The sum is infinite, not NaN; the other elements are divided by it."""
    x, r = np.ones((1, 32)), np.zeros((1, 32))
    r[0, 3] = -np.inf
    h, y = oracle.rmsnorm_ref(x, r)
    assert h[0, 3] == -np.inf and np.array_equal(np.delete(h, 3), np.ones(31))
    assert np.isnan(y[0, 3]) and not np.delete(y, 3).any()
