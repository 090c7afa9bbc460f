"""Pins of the MXFP4 oracle against the format's own tables, on the CPU."""

import numpy as np
import pytest

import oracle


def test_e2m1_values_and_round_trip():
    c = np.arange(16)
    v = oracle.e2m1_decode(c)
    assert v[:8].tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert (v[8:] == -v[:8]).all() and np.signbit(v[8])
    assert np.array_equal(oracle.e2m1_encode(v), c)


def test_e2m1_ties_go_to_the_even_code_and_large_values_saturate():
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert oracle.e2m1_encode(mids).tolist() == [0, 2, 2, 4, 4, 6, 6]
    up, down = np.nextafter(mids, 9.0), np.nextafter(mids, 0.0)
    assert oracle.e2m1_encode(up).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert oracle.e2m1_encode(down).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert oracle.e2m1_encode(np.array([7.0, 1e30, np.inf, -np.inf, -6.5])).tolist() == [7, 7, 7, 15, 15]


@pytest.mark.parametrize("amax,code", [(0.0, 0), (1.0, 125), (1.99, 125), (2.0, 126), (4.0, 127), (6.0, 127),
                                       (2.0**-125, 0), (2.0**-124, 1), (2.0**-133, 0), (3.38e38, 252),
                                       (np.inf, 255), (np.nan, 255)])
def test_scale_codes(amax, code):
    assert int(oracle.fp4_scale_code(amax)) == code


def test_quantize_bounds_the_error_by_the_formats_half_steps():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 96))
    codes, scales = oracle.quantize_fp4(x)
    v = oracle.dequantize_fp4(codes, scales)
    step = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=-1)
    a = np.abs(x) / step
    # Half a step below 6 (steps .5, 1, 2), the saturation above.
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0))
    assert (np.abs(v - x) <= np.maximum(half, a - 6) * step).all()
    assert (a < 8).all()


def test_slab_places_every_group():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (19, 160)).astype(np.uint8)
    scales = rng.integers(0, 255, (19, 5)).astype(np.uint8)
    q, s = oracle.fp4_slab(codes, scales)
    assert q.shape == (2, 16, 4, 16, 16) and s.shape == (2, 256, 4)
    for r in (0, 15, 16, 18):
        for k in (0, 31, 32, 127, 128, 159):
            byte = q[k // 128, r // 16, (k % 128) // 32, r % 16, (k % 32) // 2]
            assert (byte >> (4 * (k % 2))) & 15 == codes[r, k]
            assert s[k // 128, r, (k % 128) // 32] == scales[r, k // 32]
    assert not q[1, :, 1:].any() and not s[1, :, 1:].any() and not s[:, 19:].any()


def test_rmsnorm_ref_is_the_formula():
    x = np.array([[3.0, 4.0] * 16])
    h, y = oracle.rmsnorm_ref(x, eps=0.0)
    assert np.array_equal(h, x)
    assert np.allclose(y, x / np.sqrt(12.5), rtol=2.0**-8)
    h, y = oracle.rmsnorm_ref(x, residual=x, gain=np.full(32, 2.0), eps=0.0)
    assert np.array_equal(h, 2 * x)
    assert np.allclose(y, 2 * x / np.sqrt(12.5), rtol=2.0**-8)
