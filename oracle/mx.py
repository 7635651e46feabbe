"""Microscaled (MX) tensors: one power-of-two scale per 32 columns of a row.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definition (include/lq_mx.h), computed here in float64 from the element
formats' value lists, with no bit manipulation of the inputs:
  * grid of E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6; grid of E4M3: m 2^-9 for m < 8,
    (8 + m) 2^(e - 10) for e = 1..15, m < 8, without the last (448 is largest);
  * block scale 2^e, e the smallest integer in [-127, 127] with
    amax <= largest 2^e, stored as e + 127; a block with a non-finite element
    is stored as 255 with zero codes;
  * element code: index of the nearest grid value of |x| 2^-e (a tie goes to
    the even index), sign bit on top.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
FORMATS = ("fp4", "fp8")

_FP4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_FP8 = np.array([m * 2.0**-9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
GRID = {"fp4": _FP4, "fp8": _FP8}


def padded(cols):
    return -(-cols // BLOCK) * BLOCK


def mx_quantize(X, fmt):
    """(codes, scales) as stored: uint8 rows x (padded / 2 or padded), rows x padded / 32."""
    X = np.asarray(X, np.float64)
    rows, cols = X.shape
    kp = padded(cols)
    x = np.zeros((rows, kp))
    x[:, :cols] = X
    x = x.reshape(rows, kp // BLOCK, BLOCK)
    grid = GRID[fmt]
    fin = np.isfinite(x).all(-1)
    x = np.where(fin[..., None], x, 0.0)
    amax = np.abs(x).max(-1)
    e = np.full(amax.shape, 127)
    for t in range(126, -128, -1):  # smallest exponent that still fits
        e = np.where(amax <= grid[-1] * 2.0**t, t, e)
    a = np.abs(x) * 2.0 ** (-e[..., None].astype(np.float64))
    lo = np.searchsorted(grid, a, side="right") - 1
    hi = np.minimum(lo + 1, len(grid) - 1)
    dl, dh = a - grid[lo], grid[hi] - a
    idx = np.where((dh < dl) | ((dh == dl) & (lo % 2 == 1)), hi, lo)
    idx = np.where(hi == lo, lo, idx)
    sign = np.signbit(x).astype(np.int64)
    scales = np.where(fin, e + 127, 255).astype(np.uint8)
    if fmt == "fp8":
        codes = np.where(fin[..., None], idx | (sign << 7), 0).astype(np.uint8).reshape(rows, kp)
    else:
        c = np.where(fin[..., None], idx | (sign << 3), 0).astype(np.uint8).reshape(rows, kp)
        codes = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    return codes, scales


def mx_dequantize(codes, scales, fmt, cols):
    """Element values, float64, rows x cols (NaN in blocks of scale 255 and for E4M3 NaN codes)."""
    codes = np.asarray(codes)
    if fmt == "fp8":
        table = np.concatenate([_FP8, [np.nan]])
        table = np.concatenate([table, -table])
        v = table[codes]
    else:
        table = np.concatenate([_FP4, -_FP4])
        v = np.stack([table[codes & 15], table[codes >> 4]], -1).reshape(codes.shape[0], -1)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * np.repeat(s, BLOCK, 1))[:, :cols]
