"""The attention kernels that only larger batches reach, at ordinary sizes, against the
fp64 oracle. Each test first asserts (attn_shapes.py) which kernel and which search for
a tile its sizes take. Bounds: attn_helpers.py."""

import functools

import numpy as np
import pytest
import torch

import attn_shapes
import chunked_gated_delta_rule_amd as gdn
from attn_helpers import DEV, TYPES, Cache, check_attention, cu_of, f64, normal, on

pytestmark = pytest.mark.gpu


def lookup(n, splits):
    """How a work-group finds its tile among n sequences."""
    if splits > 1:
        return "in order"
    return "one" if n == 1 else "longest first" if n <= attn_shapes.K["kMostTiled"] else "search"


def check_shape(cfg, keys, waves, splits, how):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    s = attn_shapes.shape(cfg, keys, cus)
    assert (s.waves, s.splits > 1, lookup(cfg.n_max, s.splits)) == (waves, splits, how), s
    if keys == attn_shapes.PAGES:
        assert not attn_shapes.streams(cfg)


def sampled(lens, step):
    """(sequence, row) pairs: every step-th packed row and each sequence's last one."""
    cu = cu_of(lens)
    rows = sorted({*range(0, int(cu[-1]), step), *(int(x) - 1 for x in cu[1:])} - {-1})
    seq = np.searchsorted(cu[1:], rows, side="right")
    return [(int(s), r - int(cu[s])) for s, r in zip(seq, rows)]


def check_rows(o, q, cu, keys_of, lens, full, t, step):
    """o's sampled rows against the oracle; all rows finite."""
    assert o.isfinite().all()
    for s, r in sampled(lens, step):
        seen = full[s] - lens[s] + r + 1
        at = int(cu[s]) + r
        k, v = keys_of(s)
        check_attention(o[at:at + 1], f64(q[at:at + 1]), k[:seen], v[:seen], q.shape[2] ** -0.5, t)


def uneven(n, most, seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    return [int(x) for x in rng.integers(0, most + 1, n)]


ROWS = [
    # new tokens, older keys of each; h, hkv, d; waves, whether keys are split, search; every how many rows
    ([4096], 0, 32, 8, 128, 8, False, "one", 301),
    ([2500, 1700], 0, 16, 4, 128, 8, False, "longest first", 211),
    ([2500, 0, 3800], 70, 16, 2, 128, 8, False, "longest first", 311),
    ([2300], 0, 24, 8, 128, 8, False, "one", 151),
    ([3001], 0, 16, 2, 256, 8, False, "one", 211),
    ([1500, 900, 1301], 33, 16, 2, 256, 8, False, "longest first", 251),
    ([600, 1100], 0, 32, 8, 128, 4, False, "longest first", 97),
    (uneven(100, 60, 1), 0, 8, 2, 128, 4, False, "longest first", 29),
    (uneven(100, 60, 2), 9, 8, 2, 256, 8, False, "longest first", 29),
    (uneven(256, 31, 3), 0, 4, 4, 128, 4, False, "longest first", 37),
    (uneven(300, 40, 4), 0, 8, 2, 128, 4, False, "search", 53),
    (uneven(300, 40, 5), 21, 6, 2, 256, 8, False, "search", 53),
    ([1000], 0, 16, 4, 128, 8, True, "in order", 83),
    (uneven(70, 9, 6), 700, 2, 1, 128, 8, True, "in order", 11),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lens,past,h,hkv,d,waves,split,how,step", ROWS)
def test_prompts(t, lens, past, h, hkv, d, waves, split, how, step):
    full = [x + past for x in lens]
    T, Tk, n = sum(lens), sum(full), len(lens)
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, tk_max=Tk)
    check_shape(cfg, attn_shapes.ROWS, waves, split, how)
    q = normal(1, T, h, d, dtype=t, scale=2.0)
    k, v = (normal(i, Tk, hkv, d, dtype=t) for i in (2, 3))
    cu, cuk = cu_of(lens), cu_of(full)
    print(f"prompts {t} n={n} T={T} past={past} h={h} hkv={hkv} d={d}", flush=True)
    args = [x.to(DEV) for x in (q, k, v)]
    o = gdn.causal_attention(*args, on(cu), on(cuk))
    kd, vd = f64(k), f64(v)
    check_rows(o, q, cu, lambda s: (kd[cuk[s]:cuk[s + 1]], vd[cuk[s]:cuk[s + 1]]), lens, full, t, step)
    assert torch.equal(o, gdn.causal_attention(*args, on(cu), on(cuk)))  # the same bits again


PAGED = [
    # new tokens, older keys of each; h, hkv, d, page; waves, whether keys are split, search; step
    ([4096], 0, 32, 8, 128, 64, 8, False, "one", 401),
    ([2300, 2600], 500, 16, 4, 128, 16, 8, False, "longest first", 311),
    ([2048], 1000, 24, 2, 256, 32, 8, False, "one", 211),
    (uneven(100, 60, 7), 30, 8, 1, 128, 16, 4, False, "longest first", 31),
    (uneven(100, 40, 8), 10, 16, 2, 256, 128, 8, False, "longest first", 31),
    ([4 + i % 12 for i in range(300)], 25, 8, 1, 128, 16, 4, False, "search", 61),
    ([4 + i % 12 for i in range(280)], 25, 16, 2, 256, 32, 8, False, "search", 61),
    ([60, 3, 45], 900, 8, 1, 256, 16, 8, True, "in order", 7),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lens,past,h,hkv,d,page,waves,split,how,step", PAGED)
def test_prompts_over_pages(t, lens, past, h, hkv, d, page, waves, split, how, step):
    full = [x + past for x in lens]
    T, n = sum(lens), len(lens)
    c = Cache(full, hkv, d, page, t, 40, extra_cols=0)
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=c.n_pages, max_pages=c.cols)
    check_shape(cfg, attn_shapes.PAGES, waves, split, how)
    q = normal(1, T, h, d, dtype=t, scale=2.0)
    cu = cu_of(lens)
    print(f"prompts over pages {t} n={n} T={T} past={past} h={h} hkv={hkv} d={d}", flush=True)
    args = (q.to(DEV), c.k.to(DEV), c.v.to(DEV), on(cu), on(np.array(full, np.int32)), on(c.table))
    o = gdn.paged_attention(*args)
    check_rows(o, q, cu, functools.lru_cache(None)(c.rows), lens, full, t, step)
    assert torch.equal(o, gdn.paged_attention(*args))


@pytest.mark.parametrize("new,full,h,hkv,d,past", [
    ([1] * 70, [4400] * 70, 4, 2, 128, True),                # 315 MB, each key read by one row tile
    ([1] * 70, [2100] * 70, 4, 2, 128, False),               # 151 MB
    ([300] + [1] * 49, [9000] + [500] * 49, 8, 2, 256, False),   # 69 MB, a part of it by 38 tiles: 759
    ([150] + [1] * 69, [3000] + [300] * 69, 16, 8, 128, False),  # 97 MB, by 19: 348; more than 64 sequences
    ([60] + [1] * 69, [100] + [2100] * 69, 8, 4, 128, False),    # 298 MB, little of it by several
])
def test_streamed_keys_go_past_the_caches_only_if_read_once(new, full, h, hkv, d, past):
    """Not temporal loads are for keys that the caches could not hold and one row tile
    reads; the choice is left behind the prefix's length in the workspace."""
    t, page, n = torch.bfloat16, 16, len(new)
    need = -(-max(full) // page)
    table = np.arange(n * need, dtype=np.int32).reshape(n, need) % 64  # pages shared: any keys do
    cfg = gdn.make_attn_config(sum(new), n, h, hkv, d, t, page_size=page, n_pages=64, max_pages=need)
    assert attn_shapes.streams(cfg) and not attn_shapes.shares(cfg)
    q = torch.ones(sum(new), h, d, dtype=t, device=DEV)
    kp, vp = (normal(i, 64, hkv, page, d, dtype=t).to(DEV) for i in (2, 3))
    ws = torch.full((gdn.gdn_attn_workspace_size(cfg),), 0x55, dtype=torch.uint8, device=DEV)
    o = torch.empty_like(q)
    gdn.gdn_attn_paged(cfg, q, kp, vp, on(cu_of(new)), on(np.array(full, np.int32)), on(table), None,
                       o, ws)
    assert o.isfinite().all()
    assert ws[:8].view(torch.int32).tolist() == [0, int(past)]
