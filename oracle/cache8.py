"""fp64 reference of the 8-bit cache and of rotations by positions of several axes,
written from their definitions in include/gdn.h with NumPy: code by code, block by
block, nothing shared with the HIP library.
"""

from __future__ import annotations

import numpy as np

BLOCK = 16
# the largest number of four significant bits of each 16-bit type
TOP = {"bfloat16": 1.875 * 2.0 ** 127, "float16": 61440.0}


def _all_values():
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        if c & 127 == 127:
            v = np.nan
        out.append(-v if c & 128 else v)
    return np.array(out)


VALUES = _all_values()       # of every code
GRID = VALUES[:127]          # the finite ones from 0 on


def encode(x):
    """Codes nearest to x (ties to the even code; NaN: 127), |x| at most 448."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    assert np.all(a <= 448.0)
    hi = np.searchsorted(GRID, a)          # GRID[hi - 1] < a <= GRID[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isnan(x), 127, c | np.where(np.signbit(x), 128, 0))
    return c.astype(np.uint8)


def least_scale(a):
    """The least e >= 15 with a <= 448 * 2^(e - 127)."""
    e = 15
    while a > 448.0 * 2.0 ** (e - 127):
        e += 1
    return e


def scale_value(e):
    e = np.asarray(e, np.float64)
    return np.where(e == 255, np.nan, 2.0 ** (e - 127))


def values(codes, scales):
    """Numbers of a pool: codes [pages, hkv, size, d], scales [pages, hkv, size / 16]."""
    return VALUES[codes] * np.repeat(scale_value(scales), BLOCK, axis=2)[..., None]


def append(codes, scales, table_row, first, x, top):
    """Writes rows x [n, hkv, d] of positions first, first + 1, ... of one sequence into
    the pool, in place; positions without a page are left out."""
    pages, hkv, size, _ = codes.shape
    n = len(x)
    for block in range(first // BLOCK, (first + n - 1) // BLOCK + 1):
        places = [p for p in range(block * BLOCK, block * BLOCK + BLOCK) if first <= p < first + n]
        start = block * BLOCK
        if start < 0 or start // size >= len(table_row):
            continue
        page = int(table_row[start // size])
        if not 0 <= page < pages:
            continue
        row, b = start % size, start % size // BLOCK
        had = places[0] - start
        for h in range(hkv):
            y = np.array([x[p - first, h] for p in places], np.float64)
            fine = np.isfinite(y)
            y = np.where(fine, np.clip(y, -top, top), np.nan)
            e = least_scale(np.abs(y[fine]).max() if fine.any() else 0.0)
            if had:
                old = int(scales[page, h, b])
                e = max(e, old)
                if e > old:
                    was = VALUES[codes[page, h, row:row + had]]
                    codes[page, h, row:row + had] = encode(was * 2.0 ** (old - e))
            scales[page, h, b] = e
            codes[page, h, row + had:row + had + len(places)] = encode(y * 2.0 ** (127 - e))


def norm_rope_axes(x, w, positions, pair_axis, inv_freq, eps, interleaved=False, rot_scale=1.0):
    """x [T, heads, d]; positions [axes, T]; pair i turned by positions[pair_axis[i]] *
    inv_freq[i]. Returns (y, a) as attention.norm_rope does."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y, mag = x.copy(), np.abs(x)
    pairs = len(inv_freq)
    for i in range(pairs):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        axis = min(max(int(pair_axis[i]), 0), len(positions) - 1)
        t = np.asarray(positions[axis], np.float64) * np.float64(inv_freq[i])
        c, s = rot_scale * np.cos(t)[:, None], rot_scale * np.sin(t)[:, None]
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = np.abs(a * c) + np.abs(b * s)
        mag[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, mag
