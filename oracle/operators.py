"""Definitions, in fp64, of the MXFP4 quantiser and product and of the products
of ragged row groups with their gradients.

TEST INFRASTRUCTURE ONLY: nothing in the product path may import this module.

MXFP4 quantisation follows the OCP Microscaling Formats v1.0 rule for a block
of 32: the shared exponent is floor(log2(amax)) minus the exponent of E2M1's
largest power of two (4 = 2^2), here kept in [-125, 125] so that the scale
bytes are ones the layer's plan accepts; elements are rounded to the nearest
E2M1 value, ties to the even code, and saturate at +-6.
"""
from __future__ import annotations

import numpy as np

from .formats import E2M1_MAGNITUDES, e2m1_value, e8m0_value, pack_nibbles, unpack_nibbles


def e2m1_encode(v: np.ndarray) -> np.ndarray:
    """fp64 -> E2M1 codes: the nearest of the eight magnitudes, ties to the even
    code, |v| > 6 saturating; the sign is kept (also of a value that rounds to 0)."""
    x = np.asarray(v, dtype=np.float64)
    mags = np.asarray(E2M1_MAGNITUDES)
    mids = (mags[:-1] + mags[1:]) / 2
    a = np.abs(x)[..., None]
    # midpoint i lies between codes i and i+1: a tie goes up when i is odd
    up = np.where(np.arange(7) % 2 == 1, a >= mids, a > mids)
    return (up.sum(axis=-1) | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def mxfp4_scale_exponent(amax: np.ndarray) -> np.ndarray:
    a = np.asarray(amax, dtype=np.float64)
    _, ex = np.frexp(a)                        # a = f 2^ex, f in [0.5, 1): floor(log2 a) = ex - 1
    return np.where(a > 0, np.clip(ex - 3, -125, 125), -125)


def mxfp4_quantize(x: np.ndarray):
    """(codes [rows, cols/2], scales [rows, cols/32]) of [rows, cols]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    e = mxfp4_scale_exponent(np.abs(b).max(axis=-1))
    codes = e2m1_encode(np.ldexp(b, -e[..., None]))
    codes = np.where(bad[..., None], 0, codes).reshape(rows, cols)
    return pack_nibbles(codes), np.where(bad, 255, e + 127).astype(np.uint8)


def mxfp4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Every scale byte allowed (0xFF: NaN)."""
    v = e2m1_value(unpack_nibbles(codes))
    rows, cols = v.shape
    return (v.reshape(rows, cols // 32, 32) * e8m0_value(scales)[:, :, None]).reshape(rows, cols)


def mxfp4_matmul(a_codes, a_scales, b_codes, b_scales) -> np.ndarray:
    return mxfp4_values(a_codes, a_scales) @ mxfp4_values(b_codes, b_scales).T


def grouped_matmul(x, w, offsets, out):
    """out with rows offsets[e]..offsets[e+1]-1 replaced by x w_e^T."""
    y = np.array(out, dtype=np.float64)
    for e in range(len(w)):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        y[r] = np.asarray(x[r], np.float64) @ np.asarray(w[e], np.float64).T
    return y


def grouped_matmul_backward(dy, x, w, offsets, dx):
    """(dx with the groups' rows replaced by dy w_e, dw_e = dy_e^T x_e)."""
    gx = np.array(dx, dtype=np.float64)
    gw = np.zeros(np.shape(w))
    for e in range(len(w)):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        d = np.asarray(dy[r], np.float64)
        gx[r] = d @ np.asarray(w[e], np.float64)
        gw[e] = d.T @ np.asarray(x[r], np.float64)
    return gx, gw
