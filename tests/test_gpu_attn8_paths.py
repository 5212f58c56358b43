"""The 8-bit cache where long prompts, drafts that are taken back and keys that are not finite
lead: launch shapes of the append that only many tokens reach, each test asserting the one its
sizes take; the cache after a rejected draft; NaN in codes and scales of keys; and the call
against the 16-bit one on the same numbers. Bounds: attn_helpers.py, attn8_helpers.py."""

import numpy as np
import pytest
import torch

import attn8_shapes
import attn_shapes
import chunked_gated_delta_rule_amd as gdn
from attn8_helpers import Cache8, bytes_of, check_codes, top_of
from attn_helpers import (DEV, TYPES, check_attention, cu_of, f64, half_step, normal, on, score_error,
                          widened)
from oracle import attention, cache8

pytestmark = pytest.mark.gpu


def say(msg):
    print(msg, flush=True)


def ints(x):
    return on(np.asarray(x, np.int32))


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ---------------------------------------------------------------- append: long prompts

LONG = [
    # tokens, older ones of each sequence; h, hkv, d, page, rot, axes; parts, past the caches
    ([9007, 6600, 16, 17145], [5, 0, 33, 300], 16, 2, 256, 64, 64, 0, 3, True),
    ([14000, 1, 16003], [7, 30, 2], 32, 4, 128, 32, 128, 3, 4, True),
    ([11001, 13000], [0, 21], 16, 2, 128, 16, 66, 0, 3, False),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lens,past,h,hkv,d,page,rot,axes,parts,past_cache", LONG)
def test_append8_of_long_prompts(t, lens, past, h, hkv, d, page, rot, axes, parts, past_cache):
    """Blocks numbered eight at a time with several work-groups each, q and k stored past the
    caches or not: q and k are the 16-bit pass's, the cache is what calls of 1600 tokens (other
    parts, all blocks numbered together) leave, and sampled blocks are the oracle's."""
    T, n = sum(lens), len(lens)
    full = [a + b for a, b in zip(lens, past)]
    cu = cu_of(lens)
    need = [-(-x // page) for x in full]
    table = np.full((n, max(need)), -1, np.int32)
    order, at = np.random.Generator(np.random.PCG64(4)).permutation(sum(need)), 0
    for i, u in enumerate(need):
        table[i, :u] = order[at:at + u]
        at += u

    def cfg_of(tokens, seqs):
        return gdn.make_attn_config(tokens, seqs, h, hkv, d, t, rot_dim=rot, page_size=page, n_pages=at,
                                    max_pages=table.shape[1])

    shape = attn8_shapes.append8(cfg_of(T, n), cus())
    assert (shape.parts, shape.group, shape.past_cache) == (parts, 8, past_cache), shape
    small = attn8_shapes.append8(cfg_of(1600, 1), cus())
    assert small.whole and small.parts != parts and not small.past_cache, small
    say(f"long append8 {t} T={T} h={h} hkv={hkv} d={d} axes={axes} {shape}")

    g = torch.Generator(device=DEV).manual_seed(T + d)
    x = torch.randn(T, (h + 2 * hkv) * d, device=DEV, generator=g)
    x = (x * torch.exp2(torch.randint(-3, 4, (T, 1), device=DEV, generator=g).float())).to(t)
    w = 1.0 + 0.3 * torch.randn(d, device=DEV, generator=g)
    f = gdn.rope_inv_freq(rot).to(DEV)
    places = torch.randint(0, 100000, (axes, T), device=DEV, generator=g, dtype=torch.int32) if axes else None
    axis = (torch.arange(rot // 2) % axes).int().to(DEV) if axes else None
    # (rows that the first blocks have: any codes but NaN)
    codes = torch.randint(0, 127, (at, hkv, page, d), device=DEV, generator=g, dtype=torch.uint8)
    scales = torch.randint(110, 118, (at, hkv, page // 16), device=DEV, generator=g, dtype=torch.uint8)
    before = [codes, codes.flip(0).contiguous(), scales, scales.flip(0).contiguous()]
    whole, pieces = ([y.clone() for y in before] for _ in range(2))
    kw = dict(inv_freq=f, output_k=True, pair_axis=axis)
    q, k = gdn.append_paged_kv(x, h, on(cu), ints(full), on(table), *whole[:2], w, w, k_scales=whole[2],
                               v_scales=whole[3], positions=places, **kw)
    q2, k2 = gdn.qk_norm_rope(x, h, hkv, on(cu), w, w, f, kv_lens=None if axes else ints(full),
                              positions=places, pair_axis=axis)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    del q2, k2
    for s in range(n):
        p = past[s]
        while p < full[s]:
            end = min((p // 16 + 100) * 16, full[s])
            a, b = (int(cu[s]) + y - past[s] for y in (p, end))
            qs, ks = gdn.append_paged_kv(x[a:b], h, on(cu_of([b - a])), ints([end]), on(table[s:s + 1]),
                                         *pieces[:2], w, w, k_scales=pieces[2], v_scales=pieces[3],
                                         positions=places[:, a:b].contiguous() if axes else None, **kw)
            assert torch.equal(q[a:b], qs) and torch.equal(k[a:b], ks)
            p = end
    assert all(torch.equal(a, b) for a, b in zip(whole, pieces))

    # blocks of the oracle: each sequence's first and last, and some between
    rng = np.random.Generator(np.random.PCG64(5))
    w64, f64_, top = f64(w), f64(f), top_of(t)
    for s in range(n):
        first, last = past[s] // 16, (full[s] - 1) // 16
        for b in sorted({first, last, *rng.integers(first, last + 1, 6).tolist()}):
            lo, hi = max(16 * b, past[s]), min(16 * b + 16, full[s])
            rows = slice(int(cu[s]) + lo - past[s], int(cu[s]) + hi - past[s])
            xs = f64(x[rows]).reshape(hi - lo, -1, d)
            if axes:
                want, mag = cache8.norm_rope_axes(xs[:, h:h + hkv], w64, f64(places[:, rows]), axis.cpu().numpy(),
                                                  f64_, 1e-6)
            else:
                want, mag = attention.norm_rope(xs[:, h:h + hkv], w64, np.arange(lo, hi), f64_, 1e-6)
            page_, r0 = int(table[s, 16 * b // page]), 16 * b % page
            for i, y in ((0, want), (1, xs[:, h + hkv:])):
                one = [bytes_of(z[i][page_:page_ + 1]).copy() for z in (before, whole)]
                sc = [bytes_of(z[2 + i][page_:page_ + 1]).copy() for z in (before, whole)]
                cache8.append(one[0], sc[0], [0], r0 + lo - 16 * b, y, top)
                assert np.array_equal(sc[0][..., r0 // 16], sc[1][..., r0 // 16])
                new = slice(r0 + lo - 16 * b, r0 + hi - 16 * b)
                if i:
                    assert np.array_equal(one[0][0, :, r0:new.stop], one[1][0, :, r0:new.stop])
                else:
                    assert np.array_equal(one[0][0, :, r0:new.start], one[1][0, :, r0:new.start])
                    e = np.broadcast_to(sc[0][0, :, r0 // 16], (hi - lo, hkv))
                    check_codes(one[1][0, :, new].transpose(1, 0, 2), e, np.clip(y, -top, top), mag)
    torch.cuda.empty_cache()


def test_append8_of_the_most_tokens_and_sequences_gives_q_and_k():
    """t_max = 2^24 rows and n_max = 16384 sequences, most of them without a page: q and k of every
    row are the 16-bit pass's."""
    t, d, h, hkv, page = torch.bfloat16, 128, 1, 1, 256
    T, n = gdn.GDN_T_MAX_LIMIT, gdn.GDN_N_MAX_LIMIT
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t)
    shape = attn8_shapes.append8(cfg, cus())
    assert shape.group == 8 and shape.parts == 1 and shape.past_cache
    say(f"append8 of {T} rows, {n} sequences {shape}")
    cu = np.linspace(0, T, n + 1).astype(np.int64)
    x = torch.randint(-2 ** 15, 2 ** 15, (T, 3 * d), device=DEV, dtype=torch.int16).view(t)
    x = torch.where(x.isfinite(), x, torch.ones((), dtype=t, device=DEV))
    f, w = gdn.rope_inv_freq(64).to(DEV), torch.full((d,), 1.5, device=DEV)
    table = np.full((n, 1), -1, np.int32)
    table[-2:, 0] = 1, 0
    kv = np.diff(cu) - 700  # the first rows' positions are below zero
    pools = [torch.zeros(2, hkv, page, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros(2, hkv, page // 16, dtype=torch.uint8, device=DEV) for _ in range(2)]
    cud, kvd = on(cu.astype(np.int32)), ints(kv)
    q, k = gdn.append_paged_kv(x, h, cud, kvd, on(table), *pools, w, w, f, output_k=True,
                               k_scales=scales[0], v_scales=scales[1])
    q2, k2 = gdn.qk_norm_rope(x, h, hkv, cud, w, w, f, kvd)
    assert torch.equal(q.view(torch.int16), q2.view(torch.int16))
    assert torch.equal(k.view(torch.int16), k2.view(torch.int16))
    assert all(p.any(-1).sum() == 2 * 256 for p in pools)
    del x, q, k, q2, k2
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- append: drafts that are taken back

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("had", [5, 14, 16])
def test_append8_after_a_rejected_draft(t, d, had):
    """Of eight draft tokens three are accepted; the fifth was large. Its mark on the accepted
    rows is less than the smallest step of the block's grown scale, and the block put back as it
    was takes it away to the bit (one that begins with a draft token begins anew by itself)."""
    h, hkv, page, draft, keep, more = 2, 2, 32, 8, 3, 2
    c = Cache8([had], hkv, d, page, t, 31, extra_cols=2)
    c.table[0, :2] = np.random.Generator(np.random.PCG64(1)).permutation(c.n_pages)[:2]
    x = normal(32, had + draft + more, (h + 2 * hkv) * d, dtype=t)
    x[had + 4] *= 1000.0
    say(f"rejected draft {t} d={d} had={had}")

    def append(pools, rows, kv):
        y = x[rows].to(DEV)
        gdn.append_paged_kv(y, h, on(cu_of([len(y)])), ints([kv]), on(c.table), *pools[:2],
                            k_scales=pools[2], v_scales=pools[3])

    def start():
        pools = [p.view(torch.uint8) for p in c.on()]
        append(pools, slice(0, had), had)
        return pools

    accepted, later = slice(had, had + keep), slice(had + draft, None)
    end = had + keep + more
    plain = start()  # the draft never was
    append(plain, accepted, had + keep)
    append(plain, later, end)
    marked = start()
    append(marked, slice(had, had + draft), had + draft)
    append(marked, later, end)
    undone = start()
    page_, row = int(c.table[0, had // page]), had % page // 16 * 16
    blocks = [p[page_, :, row:row + 16] for p in undone[:2]] + [p[page_, :, row // 16] for p in undone[2:]]
    saved = [b.clone() for b in blocks]
    append(undone, slice(had, had + draft), had + draft)
    for b, s in zip(blocks, saved):
        b.copy_(s)
    append(undone, accepted, had + keep)
    append(undone, later, end)

    def rows_of(pools):
        c.k, c.v, c.ks, c.vs = (bytes_of(p) for p in pools)
        return c.rows(0, end), [np.stack([e[c.table[0, p // page], :, p % page // 16] for p in range(end)])
                                for e in (c.ks, c.vs)]

    (pk, pv), _ = rows_of(plain)
    (uk, uv), _ = rows_of(undone)
    assert np.array_equal(pk, uk) and np.array_equal(pv, uv)
    (mk, mv), es = rows_of(marked)
    differ = False
    for a, b, e in zip((pk, pv), (mk, mv), es):
        # In steps of the smallest kind by the grown scale: a row that was there is off by half a
        # step. An accepted row has its nearest multiple of a step, half a step off, where the
        # step is larger than that of the number nearest to it alone, which is at most half a step
        # apart (from four steps on; a quarter off): three quarters in all.
        step = np.exp2(e.astype(np.float64) - 136.0)[..., None]
        old = slice(0, had + keep)
        assert np.all(np.abs(a - b)[old] <= 0.75 * step[old])
        assert np.all(e[had + 4] >= 127)  # the large token's scale stays
        differ = differ or not np.array_equal(a, b)
    assert differ


# ---------------------------------------------------------------- attention: keys that are not finite

NAN = [
    # where; new tokens, tokens in all; h, hkv, d, page, shared; whether keys are streamed
    ("tokens", [1, 1], [9000, 700], 8, 2, 128, 16, 0, True),
    ("tokens", [5, 3], [300, 77], 4, 2, 256, 32, 0, True),
    ("tokens", [1, 2, 1], [900, 950, 1200], 16, 2, 256, 16, 700, True),
    ("prefix", [1, 2, 1], [900, 950, 1200], 16, 2, 256, 16, 700, True),
    ("tokens", [300, 120], [700, 333], 8, 2, 128, 16, 0, False),
    ("tokens", [140], [4000], 4, 2, 256, 64, 0, False),
    ("tokens", [60], [3000], 8, 2, 128, 128, 0, False),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("what", ["code", "scale"])
@pytest.mark.parametrize("where,new,full,h,hkv,d,page,shared,streams", NAN)
def test_paged8_of_keys_that_are_not_finite(t, what, where, new, full, h, hkv, d, page, shared, streams):
    """NaN in a key's code, or 255 as the scale of a block of keys, of one key head, among the
    last sequence's new tokens or in the prefix of all: the rows that see such a key are NaN in
    that head's group, all others the oracle's; a key that the row's mask hides does nothing."""
    c = Cache8(full, hkv, d, page, t, 7, shared)
    n, T, last = len(new), sum(new), len(new) - 1
    q = normal(8, T, h, d, dtype=t)
    rows = [c.rows(s) for s in range(n)]  # before
    at = 5 if where == "prefix" else full[last] - 1 - new[last] // 2
    if what == "code":
        c.k[c.table[last, at // page], 0, at % page, 3] = 255
        first = at
    else:
        c.ks[c.table[last, at // page], 0, at % page // 16] = 255
        first = at // 16 * 16
    table = widened(c.table, -(-(1 << 28) // (2 * n * hkv * d * page))) if shared else c.table
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=c.n_pages, max_pages=table.shape[1],
                               shared_max=table.shape[1] * page if shared else 0)
    assert shared or attn_shapes.streams(cfg) == streams
    say(f"NaN in keys {what} {t} {new} {full} d={d} shared={shared}")
    kp, vp, ks, vs = c.on()
    cu = cu_of(new)
    o = gdn.paged_attention(q.to(DEV), kp, vp, on(cu), ints(full), on(table), ints([shared]) if shared else None,
                            k_scales=ks, v_scales=vs)
    G = h // hkv
    for s in range(n):
        a = o[int(cu[s]):int(cu[s + 1])]
        qs, (k, v) = f64(q[int(cu[s]):int(cu[s + 1])]), rows[s]
        hit = (full[s] - new[s] + np.arange(new[s]) >= first) & (s == last or where == "prefix")
        assert a[torch.from_numpy(hit).to(DEV)][:, :G].isnan().all()
        want = attention.attend(qs, k, v, d ** -0.5)
        clean = np.broadcast_to(~hit[:, None], (new[s], h)).copy()
        clean[:, G:] = True
        pick = torch.from_numpy(clean).to(DEV)
        assert a[pick].isfinite().all()
        fixed = torch.where(pick[..., None], a, torch.from_numpy(want[0]).to(DEV).to(t))
        check_attention(fixed, qs, k, v, d ** -0.5, t, want)


# ---------------------------------------------------------------- attention: against 16-bit pages

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("new,full,h,hkv,d", [([1, 1, 1], [70, 900, 3000], 16, 2, 128),
                                              ([5, 2], [600, 77], 8, 2, 256),
                                              ([200, 130], [700, 900], 8, 2, 128),
                                              ([300], [2000], 16, 2, 256)])
def test_paged8_is_near_the_16_bit_call_row_by_row(t, new, full, h, hkv, d):
    """On the same numbers either call is off by its bound (attn_helpers.py) at most: the two
    differ by no more than both, value by value."""
    c = Cache8(full, hkv, d, 32, t, 23)
    q = normal(1, sum(new), h, d, dtype=t)
    kp, vp, ks, vs = c.on()
    say(f"8 and 16 bits row by row {t} {new} d={d}")
    cu = cu_of(new)
    batch = (on(cu), ints(full), on(c.table))
    o = gdn.paged_attention(q.to(DEV), kp, vp, *batch, k_scales=ks, v_scales=vs)
    wide = [(x.float() * s.float().repeat_interleave(16, 2)[..., None]).to(t) for x, s in ((kp, ks), (vp, vs))]
    o16 = gdn.paged_attention(q.to(DEV), *wide, *batch)
    u = half_step(t)
    for s in range(len(new)):
        a = slice(int(cu[s]), int(cu[s + 1]))
        qs, (k, v) = f64(q[a]), c.rows(s)
        want, mag, total = attention.attend(qs, k, v, d ** -0.5)
        bound = 1.01 * (u * np.abs(want) + (u + 2 * score_error(qs, k, d, d ** -0.5) + 2.0 ** -18) * mag)
        if t == torch.float16:
            bound = bound + len(k) * 2.0 ** -25 * np.abs(v).max() / total[..., None] + 2.0 ** -25
        off = np.abs(f64(o[a]) - f64(o16[a]))
        say(f"  off / bound {np.max(off / (2 * bound)):.3f}")
        assert np.all(off <= 2 * bound)
