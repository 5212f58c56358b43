"""Shared by the tests of the 8-bit cache: pools on the CPU side, and the bound that
appended codes are held to.

Values x of a token are off by fp32 arithmetic alone before they are rounded to a code
(keys: norm and rotation, 2^-17 of |a cos t| + |b sin t| as attn_helpers.py derives; values:
not at all), times a power of two, exactly. So a code's value is as near to x as the
nearest code's, but for twice that. Rows that a block had are rounded from what the
cache held: exactly the oracle's.

Attention: the numbers of the cache have four significant bits, which both 16-bit types
hold exactly as long as they are in range, so attn_helpers.py's bounds hold as they are.
"""

import numpy as np
import torch

from attn_helpers import DEV
from oracle import cache8


def top_of(t):
    return cache8.TOP[str(t).replace("torch.", "")]


def quantised(x, top):
    """Codes and scales of rows x [pages, hkv, size, d], blocks at once."""
    pages, hkv, size, d = x.shape
    y = np.clip(np.asarray(x, np.float64), -top, top).reshape(pages, hkv, size // 16, 16 * d)
    a = np.abs(y).max(-1)
    e = np.ceil(np.log2(np.maximum(a, 1e-300) / 448.0))
    e = np.where(a > 448.0 * 2.0 ** e, e + 1, e)
    e = np.clip(e + 127, 15, 247).astype(np.int64)
    codes = cache8.encode(y * (2.0 ** (127 - e))[..., None]).reshape(x.shape)
    return codes, e.astype(np.uint8)


class Cache8:
    """A paged cache for given lengths on the CPU side: random page order; heads, blocks and
    channels of unlike size; rows past a sequence's length NaN, scales of blocks without a
    row 255 (NaN). Optionally the first `shared` positions (whole pages) of all sequences in
    the same pages."""

    def __init__(self, lens, hkv, d, page, t, seed, shared=0, spare=2, extra_cols=1):
        rng = np.random.Generator(np.random.PCG64(seed))
        sp = shared // page
        used = [max(-(-n // page) - sp, 0) for n in lens]
        self.n_pages = sp + sum(used) + spare
        self.cols = max([-(-n // page) for n in lens] + [1]) + extra_cols
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), self.cols), -1, np.int32)
        at = sp
        for i, u in enumerate(used):
            row = list(order[:sp]) + list(order[at:at + u])
            self.table[i, :len(row)] = row
            at += u
        shape = (self.n_pages, hkv, page, d)
        keep = np.zeros((self.n_pages, page), bool)
        for i, n in enumerate(lens):
            p = np.arange(n)
            keep[self.table[i, p // page], p % page] = True
        some = keep.reshape(self.n_pages, page // 16, 16).any(-1)
        for name in ("k", "v"):
            size = np.exp2(rng.integers(-2, 3, (self.n_pages, hkv, page // 16)).repeat(16, 2))[..., None]
            codes, scales = quantised(rng.standard_normal(shape, np.float32) * size, top_of(t))
            codes = np.where(keep[:, None, :, None], codes, rng.choice([127, 255], shape)).astype(np.uint8)
            scales = np.where(some[:, None], scales, 255).astype(np.uint8)
            setattr(self, name, codes)
            setattr(self, name + "s", scales)
        self.lens, self.page = list(lens), page

    def on(self, dev=DEV):
        """k, v (e4m3), their scales (e8m0) on the device."""
        code = lambda x: torch.from_numpy(x).to(dev).view(torch.float8_e4m3fn)  # noqa: E731
        scale = lambda x: torch.from_numpy(x).to(dev).view(torch.float8_e8m0fnu)  # noqa: E731
        return code(self.k), code(self.v), scale(self.ks), scale(self.vs)

    def rows(self, s, n=None):
        """k and v of sequence s in 64 bits, [length, hkv, d]."""
        n = self.lens[s] if n is None else n
        p = np.arange(n)
        page, row = self.table[s, p // self.page], p % self.page
        return tuple(cache8.VALUES[c[page, :, row]] *
                     cache8.scale_value(e[page, :, row // 16])[..., None]
                     for c, e in ((self.k, self.ks), (self.v, self.vs)))


def bytes_of(x):
    return x.detach().cpu().view(torch.uint8).numpy()


def check_codes(codes, scales, x, mag):
    """Codes of rows with their scale bytes against the values x, in 64 bits."""
    s = cache8.scale_value(scales)[..., None]
    got = cache8.VALUES[codes] * s
    best = cache8.VALUES[cache8.encode(np.clip(x / s, -448.0, 448.0))] * s
    slack = 2.0 * 1.01 * 2.0 ** -17 * mag
    off, least = np.abs(got - x), np.abs(best - x)
    assert np.all(off <= least + slack), float(np.max((off - least) / np.maximum(slack, 1e-300)))
