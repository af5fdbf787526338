"""Pins of the oracle's MXFP4 quantiser and of the grouped products: nearest-value
search, closed forms and scalar loops."""
import numpy as np
import pytest

import oracle
from oracle import formats as F


def test_e2m1_encode_is_the_nearest_value_with_even_ties():
    v = np.concatenate([np.linspace(-8, 8, 4097), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -2.5, 1e9, -1e9, -0.0]])
    codes = oracle.e2m1_encode(v)
    mags = np.asarray(F.E2M1_MAGNITUDES)
    for x, c in zip(v, codes):
        d = np.abs(mags - min(abs(x), 6.0))
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else next(b for b in best if b % 2 == 0)
        assert c == want + (8 if np.signbit(x) else 0), (x, c)


def test_scale_exponent_boundaries():
    for j in range(-140, 127):
        for f, want in ((1.0, j - 2), (1.999, j - 2), (0.999, j - 3)):
            assert oracle.mxfp4_scale_exponent(f * 2.0 ** j) == np.clip(want, -125, 125)
    assert oracle.mxfp4_scale_exponent(0.0) == -125


def test_values_of_the_grid_come_back():
    """Every E2M1 value times a power of two, the block maximum 4 or 6 steps: exact."""
    mags = np.asarray(F.E2M1_MAGNITUDES)
    block = np.concatenate([mags, -mags, mags, -mags])
    for e in (-100, -3, 0, 5, 120):
        x = np.ldexp(block, e)[None, :]
        np.testing.assert_array_equal(oracle.mxfp4_values(*oracle.mxfp4_quantize(x)), x)


def test_quantisation_error_is_bounded_by_the_grid():
    """|x - q| <= 1 unit of 2^e below saturation (half the largest gap, 4..6),
    at most 2 units between 6 and 8."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 256)) * np.exp(rng.standard_normal((64, 1)) * 4)
    codes, scales = oracle.mxfp4_quantize(x)
    unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    err = np.abs(oracle.mxfp4_values(codes, scales) - x) / unit
    assert (err[np.abs(x) / unit <= 6] <= 1).all() and (err <= 2).all()
    assert (np.abs(x).reshape(64, 8, 32).max(-1) / unit[:, ::32] >= 4).all()
    assert (np.abs(x).reshape(64, 8, 32).max(-1) / unit[:, ::32] < 8).all()


def test_non_finite_blocks():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.nan, -np.inf
    codes, scales = oracle.mxfp4_quantize(x)
    np.testing.assert_array_equal(scales, [[255, 125], [125, 255]])
    assert (codes[0, :16] == 0).all() and (codes[1, 16:] == 0).all()
    v = oracle.mxfp4_values(codes, scales)
    assert np.isnan(v[0, :32]).all() and np.isnan(v[1, 32:]).all() and (v[0, 32:] == 1).all()


def test_matmul_against_scalar_loops():
    rng = np.random.default_rng(4)
    a, b = rng.integers(0, 256, (3, 32), dtype=np.uint8), rng.integers(0, 256, (2, 32), dtype=np.uint8)
    sa, sb = rng.integers(120, 131, (3, 2), dtype=np.uint8), rng.integers(120, 131, (2, 2), dtype=np.uint8)
    y = oracle.mxfp4_matmul(a, sa, b, sb)
    for i in range(3):
        for j in range(2):
            total = 0.0
            for k in range(64):
                ca, cb = (a[i, k // 2] >> (4 * (k % 2))) & 15, (b[j, k // 2] >> (4 * (k % 2))) & 15
                total += (oracle.e2m1_closed_form(int(ca)) * oracle.e2m1_closed_form(int(cb))
                          * 2.0 ** (int(sa[i, k // 32]) + int(sb[j, k // 32]) - 254))
            assert y[i, j] == pytest.approx(total, rel=1e-14)


def test_grouped_against_scalar_loops_and_differences():
    rng = np.random.default_rng(5)
    counts = [2, 0, 3, 1]
    offsets = np.concatenate([[1], 1 + np.cumsum(counts)])     # row 0 and row 7 belong to nobody
    x, w, dy = rng.standard_normal((8, 5)), rng.standard_normal((4, 3, 5)), rng.standard_normal((8, 3))
    y = oracle.grouped_matmul(x, w, offsets, np.full((8, 3), 7.0))
    dx, dw = oracle.grouped_matmul_backward(dy, x, w, offsets, np.full((8, 5), 9.0))
    want_dw = np.zeros_like(w)
    for r in range(8):
        e = next((e for e in range(4) if offsets[e] <= r < offsets[e + 1]), None)
        for n in range(3):
            assert y[r, n] == pytest.approx(7.0 if e is None else sum(w[e, n, k] * x[r, k] for k in range(5)))
            for k in range(5):
                if e is not None:
                    want_dw[e, n, k] += dy[r, n] * x[r, k]
        for k in range(5):
            assert dx[r, k] == pytest.approx(9.0 if e is None else sum(w[e, n, k] * dy[r, n] for n in range(3)))
    np.testing.assert_allclose(dw, want_dw, rtol=1e-13, atol=1e-15)
    assert (dw[1] == 0).all()
    # central differences of sum(dy * y) in a random direction (the product is linear in each argument)
    loss = lambda x, w: (dy * oracle.grouped_matmul(x, w, offsets, np.zeros((8, 3)))).sum()
    gx, _ = oracle.grouped_matmul_backward(dy, x, w, offsets, np.zeros((8, 5)))
    ux, uw, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-3
    assert (loss(x + h * ux, w) - loss(x - h * ux, w)) / (2 * h) == pytest.approx((gx * ux).sum(), rel=1e-9)
    assert (loss(x, w + h * uw) - loss(x, w - h * uw)) / (2 * h) == pytest.approx((dw * uw).sum(), rel=1e-9)
