"""Shared by the softmax-attention tests: seeded inputs, and the bounds the GPU
results are held to.

Rounding to a 16-bit type is off by at most u = eps / 2 of the value (bf16
2^-8, fp16 2^-11). The bounds count those, and fp32 arithmetic:

 norm + rotation: one rounding of the result, u |y|; before it fp32 values: the
   norm (a sum of d squares, a root, a quotient, a weight: under 2^-19 relative
   for d <= 256), the angle (rounded to 2^-25 turns, 2 pi 2^-25 < 2^-22 radians)
   and the hardware sine and cosine (2^-20 absolute), each times the pair's
   terms: 2^-17 (|a cos t| + |b sin t|) covers their sum. fp16 subnormals:
   half the smallest one, 2^-25.

 attention: one rounding of the result, u |o|; every weight rounded once to the
   16-bit type, u sum p |v|; scores summed in fp32, off by at most
   d 2^-24 sum_i |q_i k_i| scale =: e, which moves a weight, and their sum, by e
   relatively each: 2 e sum p |v|; exp2 and sums in fp32: 2^-18 sum p |v|. fp16
   weights below 2^-14 are subnormal, off by at most 2^-25 against weights that
   sum to `total` (their largest is 1): keys 2^-25 max |v| / total. Each bound is
   taken 1 % wider, for products of the terms.
"""

import numpy as np
import torch

TYPES = [torch.bfloat16, torch.float16]
DEV = "cuda:0"


def half_step(t):
    return torch.finfo(t).eps / 2


def f64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def cu_of(lens, n_max=None):
    cu = np.zeros((len(lens) if n_max is None else n_max) + 1, np.int32)
    cu[1:len(lens) + 1] = np.cumsum(lens)
    cu[len(lens) + 1:] = cu[len(lens)]
    return cu


def on(x, dev=DEV):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev)


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype)


def check_norm_rope(got, want, mag, t):
    bound = 1.01 * (half_step(t) * np.abs(want) + 2.0 ** -17 * mag) + 2.0 ** -25
    off = np.abs(f64(got) - want)
    assert np.all(off <= bound), (np.max(off / np.maximum(bound, 1e-300)))


def score_error(q, k, d, scale):
    """Largest e of a row block: d 2^-24 scale max sum |q_i k_i|."""
    if not q.size or not k.size:
        return 0.0
    H, hkv = q.shape[1], k.shape[1]
    kk = np.repeat(np.abs(k), H // hkv, axis=1)
    return d * 2.0 ** -24 * scale * max(
        float((np.abs(q[:, h]) @ kk[:, h].T).max()) for h in range(H))


def check_attention(got, q, k, v, scale, t, want=None):
    """One sequence's rows against the oracle; returns max off / bound."""
    from oracle import attention
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    d = q.shape[2]
    o, mag, total = attention.attend(q, k, v, scale) if want is None else want
    e = score_error(q, k, d, scale)
    u = half_step(t)
    bound = 1.01 * (u * np.abs(o) + (u + 2 * e + 2.0 ** -18) * mag)
    if t == torch.float16 and v.size:
        bound = bound + len(k) * 2.0 ** -25 * np.abs(v).max() / total[..., None] + 2.0 ** -25
    g = f64(got)
    assert np.all(np.isfinite(g)), "non-finite output"
    off = np.abs(g - o)
    worst = float(np.max(off / np.maximum(bound, 1e-300))) if off.size else 0.0
    assert np.all(off <= bound), worst
    return worst


class Cache:
    """A paged cache for given lengths on the CPU side: random page order, rows
    past a sequence's length poisoned with NaN, optionally the first `shared`
    positions (whole pages) of all sequences in the same pages."""

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
        self.k, self.v = normal(seed + 1, *shape, dtype=t), normal(seed + 2, *shape, dtype=t)
        keep = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for i, n in enumerate(lens):
            for p in range(n):
                keep[self.table[i, p // page], p % page] = True
        bad = ~keep[:, None, :, None]
        self.k = torch.where(bad, torch.tensor(float("nan"), dtype=t), self.k)
        self.v = torch.where(bad, torch.tensor(float("nan"), dtype=t), self.v)
        self.lens, self.page = lens, page

    def rows(self, s):
        from oracle import attention
        return (attention.gather(f64(self.k), self.table[s], self.lens[s]),
                attention.gather(f64(self.v), self.table[s], self.lens[s]))


def shared_cols(n, hkv, d, page):
    """Table columns with which n sequences of a batch are worth a pass of its own over
    a shared prefix as long as the table (256 MiB of keys and values read by them all)."""
    return -(-(1 << 28) // (4 * n * hkv * d * page))


def widened(table, cols):
    """The table with columns that name no page up to `cols`."""
    pad = np.full((table.shape[0], max(cols - table.shape[1], 0)), -1, np.int32)
    return np.concatenate([table, pad], 1)
