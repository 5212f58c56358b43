"""fp64 reference of the softmax-attention operators, written from their
definitions in include/gdn.h with NumPy: head by head, row by row, no tiling,
no running statistics and nothing shared with the HIP library.
"""

from __future__ import annotations

import numpy as np


def norm_rope(x, w, positions, inv_freq, eps, interleaved=False, rot_scale=1.0):
    """x [T, heads, d]: RMS norm with weight w [d] (None: no norm), then the pairs
    of the first 2 len(inv_freq) dims turned by position * inv_freq.

    Returns (y, a): y as defined, and |a cos t| + |b sin t| of every value, the
    magnitude that rounding errors of the pair's terms go by."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y, mag = x.copy(), np.abs(x)
    f = np.zeros(0) if inv_freq is None else np.asarray(inv_freq, np.float64)
    r = len(f)
    for i in range(r):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        t = np.asarray(positions, np.float64) * f[i]
        c, s = rot_scale * np.cos(t)[:, None], rot_scale * np.sin(t)[:, None]
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = np.abs(a * c) + np.abs(b * s)
        mag[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, mag


def positions(cu, kv_lens=None):
    """Position of every packed row."""
    out = []
    for s in range(len(cu) - 1):
        n = int(cu[s + 1] - cu[s])
        total = n if kv_lens is None else int(kv_lens[s])
        out += list(range(total - n, total))
    return np.array(out, np.float64)


def attend(q, k, v, scale):
    """Rows q [lq, H, d] on keys k, v [lk, Hkv, d]; row i sees keys 0 .. lk - lq + i.

    Returns (o, mag, total): the output, sum_c p_c |v_c| (what the rounding of
    weights goes by) and sum_c exp(s_c - max) of every row."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    lq, H, d = q.shape
    lk, hkv, _ = k.shape
    o, mag, total = np.zeros((lq, H, d)), np.zeros((lq, H, d)), np.ones((lq, H))
    for i in range(lq):
        seen = lk - lq + i + 1
        if seen <= 0:
            continue
        for h in range(H):
            j = h // (H // hkv)
            s = scale * (k[:seen, j] @ q[i, h])
            e = np.exp(s - s.max())
            total[i, h] = e.sum()
            p = e / e.sum()
            o[i, h], mag[i, h] = p @ v[:seen, j], p @ np.abs(v[:seen, j])
    return o, mag, total


def gather(pages, table_row, length):
    """The first `length` positions of one sequence: [length, Hkv, d]."""
    _, hkv, size, d = pages.shape
    rows = [pages[table_row[p // size], :, p % size] for p in range(length)]
    return np.stack(rows) if rows else np.zeros((0, hkv, d))
