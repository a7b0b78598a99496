"""fp64 oracle of MXFP4 (TEST INFRASTRUCTURE): E2M1 codes, two per byte with
the even column in the low nibble, and one E8M0 scale byte per 32 columns.

Written from the format's definition, element by element: a code's magnitude
is (-1)^sign * 2^(e-1) * (1 + m/2) for e > 0 and m/2 for e = 0; a scale byte s
is 2^(s-127), 255 is NaN.  The quantiser picks the smallest 2^k, k >= -126,
with amax <= 6 * 2^k (2^0 for zeros; NaN for a block with an infinity or a NaN)
and the nearest code, ties to the even one.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mxfp4_decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """(rows, cols/2) and (rows, cols/32) uint8 -> (rows, cols) fp64."""
    codes = np.asarray(codes, np.uint8)
    n = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(n & 8, -1.0, 1.0) * GRID[n & 7]
    s = np.asarray(scales, np.uint8).astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, np.minimum(s, 254) - 127))
    return v * np.repeat(f, 32, axis=-1)


def mxfp4_scale(amax: np.ndarray) -> np.ndarray:
    """Scale bytes of blocks with these largest magnitudes (inf or NaN: 255)."""
    amax = np.asarray(amax, np.float64)
    ok = np.isfinite(amax)
    a = np.where(ok & (amax > 0), amax, 6.0)
    k = np.ceil(np.log2(a / 6.0)).astype(np.int64)
    k = np.where(np.ldexp(6.0, k) < a, k + 1, k)
    k = np.where(np.ldexp(6.0, k - 1) >= a, k - 1, k)
    return np.where(ok, np.maximum(k, -126) + 127, 255).astype(np.uint8)


def mxfp4_encode(v: np.ndarray):
    """(rows, cols) -> codes (rows, cols/2), scales (rows, cols/32)."""
    v = np.asarray(v, np.float64)
    b = v.reshape(*v.shape[:-1], -1, 32)
    bad = ~np.all(np.isfinite(b), axis=-1)
    with np.errstate(invalid="ignore"):
        s = mxfp4_scale(np.where(bad, np.inf, np.max(np.abs(b), axis=-1)))
    k = np.where(bad, 0, s.astype(np.int64) - 127)
    a = np.where(bad[..., None], 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)))
    a = np.ldexp(a, -k[..., None])
    hi = np.clip(np.searchsorted(GRID, a, side="left"), 0, 7)     # first grid value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (hi == 0), hi, lo)
    code = np.where(bad[..., None], 0, code | (np.signbit(b) << 3)).astype(np.uint8)
    code = code.reshape(v.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s
