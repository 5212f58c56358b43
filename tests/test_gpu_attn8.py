"""GPU parity of the 8-bit cache (append, attention over its pages) and of rotations by
positions of several axes against the fp64 CPU oracle, through the C ABI. The bounds are
derived in attn_helpers.py and attn8_helpers.py."""

import functools

import numpy as np
import pytest
import torch

import chunked_gated_delta_rule_amd as gdn
from attn8_helpers import Cache8, bytes_of, check_codes, top_of
from attn_helpers import (DEV, TYPES, check_attention, check_norm_rope, cu_of, f64, normal, on,
                          widened)
from oracle import attention, cache8

pytestmark = pytest.mark.gpu
MARK = 12288.0  # exact in both types


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    gdn.load_library()  # raises if the HIP library is missing


def say(msg):
    print(msg, flush=True)


def workspace(cfg):
    return torch.full((gdn.gdn_attn_paged8_workspace_size(cfg),), 0xff, dtype=torch.uint8, device=DEV)


def ints(x):
    return on(np.asarray(x, np.int32))


# ---------------------------------------------------------------- positions of several axes

ROTS = [(128, 128, False, 3), (128, 128, True, 3), (128, 2, False, 2), (128, 66, False, 4),
        (128, 64, True, 1), (256, 64, False, 3), (256, 256, False, 16), (256, 250, False, 3),
        (256, 10, True, 2), (256, 256, True, 3)]


def places_of(T, axes, seed, most=100000):
    rng = np.random.Generator(np.random.PCG64(seed))
    p = rng.integers(-50, most, (axes, T)).astype(np.int32)
    p[:, 0] = 2_000_000_000
    return p


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,rot,inter,axes", ROTS)
def test_norm_rope_axes(t, d, rot, inter, axes):
    lens, h, hkv, spare = [3, 0, 1, 17], 6, 2, 4
    T = sum(lens)
    cu = cu_of(lens, len(lens) + 1)
    qkv = normal(d + rot, T + spare, (h + 2 * hkv) * d, dtype=t)
    qw, kw = normal(1, d, dtype=torch.float32), normal(2, d, dtype=torch.float32)
    f = gdn.rope_inv_freq(rot, 10000.0)
    places = places_of(T + spare, axes, rot)
    axis = np.random.Generator(np.random.PCG64(3)).integers(0, axes, rot // 2).astype(np.int32)
    say(f"norm_rope_axes {t} d={d} rot={rot} inter={inter} axes={axes}")
    cfg = gdn.make_attn_config(T + spare, len(lens) + 1, h, hkv, d, t, rot_dim=rot,
                               rot_interleaved=inter, rot_scale=1.25, eps=1e-5)
    q = torch.full((T + spare, h, d), MARK, dtype=t, device=DEV)
    k = torch.full((T + spare, hkv, d), MARK, dtype=t, device=DEV)
    gdn.gdn_qk_norm_rope_axes(cfg, qkv.to(DEV), qw.to(DEV), kw.to(DEV), f.to(DEV), on(places),
                              on(axis), on(cu), q, k)
    x = f64(qkv)[:T].reshape(T, h + 2 * hkv, d)
    for got, part, w in ((q, x[:, :h], qw), (k, x[:, h:h + hkv], kw)):
        want, mag = cache8.norm_rope_axes(part, f64(w), places[:, :T], axis, f64(f), 1e-5, inter, 1.25)
        check_norm_rope(got[:T], want, mag, t)
        assert (got[T:] == MARK).all()  # rows behind the last sequence


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (256, 64, True), (128, 34, False)])
def test_axes_of_equal_positions_are_the_plain_rotation(t, d, rot, inter):
    """Every axis at a token's place in its sequence: the same bits as without axes, q and k
    and the pages; many tokens, several of them per work-group."""
    lens, h, hkv, page = [700, 1, 0, 4300, 77], 4, 2, 32
    T, n = sum(lens), len(lens)
    kv = [x + 5 * i for i, x in enumerate(lens)]
    cu = cu_of(lens)
    qkv = normal(4, T, (h + 2 * hkv) * d, dtype=t).to(DEV)
    w, f = normal(5, d, dtype=torch.float32).to(DEV), gdn.rope_inv_freq(rot).to(DEV)
    need = [-(-x // page) for x in kv]
    table = np.full((n, max(need)), -1, np.int32)
    at = 0
    for i, u in enumerate(need):
        table[i, :u] = range(at, at + u)
        at += u
    places = on(np.repeat(attention.positions(cu, kv)[None], 3, 0).astype(np.int32))
    axis = gdn.rope_pair_axis([rot // 2 - 2, 1, 1], True, device=DEV) if rot > 4 else None
    pools = [torch.full((at, hkv, page, d), MARK, dtype=t, device=DEV) for _ in range(4)]
    say(f"axes as one {t} d={d} rot={rot}")
    args = (qkv, h, on(cu), ints(kv), on(table))
    kw = dict(interleaved=inter, output_k=True)
    one = gdn.append_paged_kv(*args, *pools[:2], w, w, f, **kw)
    many = gdn.append_paged_kv(*args, *pools[2:], w, w, f, positions=places, pair_axis=axis, **kw)
    assert torch.equal(one[0], many[0]) and torch.equal(one[1], many[1])
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    q, k = gdn.qk_norm_rope(qkv, h, hkv, on(cu), w, w, f, interleaved=inter, positions=places,
                            pair_axis=axis)
    assert torch.equal(q, one[0]) and torch.equal(k, one[1])


@pytest.mark.parametrize("t", TYPES)
def test_append_axes_places_rows_by_kv_lens(t):
    """The pages go by kv_lens, the angles by the positions; axes outside their range count
    as the nearest; rows of qkv inside wider ones."""
    d, h, hkv, page, rot = 128, 2, 1, 16, 96
    lens, kv = [20, 3], [33, 3]
    T = sum(lens)
    wide = normal(3, T, 5 * d, dtype=t).to(DEV)
    qkv = wide[:, d:]
    table = np.array([[4, 0, 2], [1, -1, -1]], np.int32)
    places, axis = places_of(T, 2, 9), np.arange(-3, rot // 2 - 3).astype(np.int32)
    f = gdn.rope_inv_freq(rot)
    kp, vp = (torch.full((5, hkv, page, d), MARK, dtype=t, device=DEV) for _ in range(2))
    say(f"append_axes {t}")
    q, k = gdn.append_paged_kv(qkv, h, on(cu_of(lens)), ints(kv), on(table), kp, vp,
                               inv_freq=f.to(DEV), positions=on(places), pair_axis=on(axis),
                               output_k=True)
    x = f64(qkv).reshape(T, 4, d)
    for got, part in ((q, x[:, :h]), (k, x[:, h:h + 1])):
        want, mag = cache8.norm_rope_axes(part, None, places, axis, f64(f), 1e-6)
        check_norm_rope(got, want, mag, t)
    row = 0
    seen = torch.zeros(5, page, dtype=torch.bool)
    for s in range(2):
        for p in range(kv[s] - lens[s], kv[s]):
            at = table[s, p // page], p % page
            seen[at] = True
            assert torch.equal(kp[at[0], :, at[1]], k[row])
            assert torch.equal(vp[at[0], :, at[1]], qkv.view(T, 4, d)[row, 3:])
            row += 1
    assert (kp.transpose(1, 2)[~seen] == MARK).all()


# ---------------------------------------------------------------- append

APPEND = [
    # d, page, interleaved, rot_dim, axes, norm
    (128, 16, False, 128, 0, True), (256, 64, True, 64, 0, True), (128, 256, False, 30, 0, True),
    (256, 32, False, 256, 3, True), (128, 32, True, 128, 2, True), (256, 16, False, 250, 0, True),
    (128, 64, False, 0, 0, False), (256, 128, False, 0, 0, False),
]


def run_append(cfg, c, qkv, w, f, cu, kv, q, k, places=None, axis=None):
    pools = c.on()
    gdn.gdn_kv_append8(cfg, qkv, w, w, f, places, axis, on(cu), ints(kv), on(c.table), q, k, *pools)
    return pools


def check_append(c, pools, x, lens, kv, cu, want_k, mag_k, top):
    """Pools after appending rows x [T, heads, d]'s v (exact) and keys that the oracle has as
    want_k, against the pools c as they were."""
    hkv, d = want_k.shape[1:]
    for name, got, got_s, rows, mag in (("k", pools[0], pools[2], want_k, mag_k),
                                        ("v", pools[1], pools[3], x[:, -hkv:], None)):
        got, got_s = bytes_of(got), bytes_of(got_s)
        codes, scales = getattr(c, name).copy(), getattr(c, name + "s").copy()
        for s in range(len(lens)):
            if lens[s]:
                cache8.append(codes, scales, c.table[s], kv[s] - lens[s], rows[cu[s]:cu[s + 1]], top)
        # (an fp32 key that lies as near as 2^-17 to a power of two times 448 would have
        # either scale: none of these seeds has one)
        assert np.array_equal(got_s, scales)
        nan = np.isnan(cache8.VALUES[codes])
        assert np.array_equal(np.isnan(cache8.VALUES[got]), nan)
        if mag is None or not mag.any():
            assert np.array_equal(got[~nan], codes[~nan])
            continue
        new = np.zeros(codes.shape[:1] + codes.shape[2:3], bool)
        for s in range(len(lens)):
            for i, p in enumerate(range(kv[s] - lens[s], kv[s])):
                page, r = c.table[s, p // c.page], p % c.page
                new[page, r] = True
                e = scales[page, :, r // 16]
                y = np.clip(rows[cu[s] + i], -top, top)
                check_codes(got[page, :, r], e, y, mag[cu[s] + i])
        old = ~new[:, None, :, None] & ~nan
        assert np.array_equal(got[old], codes[old])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,page,inter,rot,axes,norm", APPEND)
def test_append8(t, d, page, inter, rot, axes, norm):
    """Codes and scales of the blocks that get tokens, rows that were there rounded to a new
    scale, everything else in the pools as it was; q and k as the 16-bit pass has them."""
    lens, h, hkv = [1, 0, 37, 5, 1, 1, 16, 2, 1], 6, 3
    kv = [1, 3, 37 + 30, 5 + page - 2, 300, 16, 48, 33, 63]
    T, n = sum(lens), len(lens)
    c = Cache8(kv, hkv, d, page, t, 11)
    cu = cu_of(lens)
    size = 2.0 ** np.random.Generator(np.random.PCG64(2)).integers(-3, 5, (T + 3, 1))
    qkv = (normal(12, T + 3, (h + 2 * hkv) * d, dtype=torch.float32) * torch.from_numpy(size)).to(t)
    w = normal(13, d, dtype=torch.float32) if norm else None
    f = gdn.rope_inv_freq(rot) if rot else None
    places = places_of(T + 3, axes, 5) if axes else None
    axis = (np.arange(rot // 2) % axes).astype(np.int32) if axes else None
    say(f"append8 {t} d={d} page={page} rot={rot} axes={axes}")
    cfg = gdn.make_attn_config(T + 3, n, h, hkv, d, t, rot_dim=rot, rot_interleaved=inter,
                               page_size=page, n_pages=c.n_pages, max_pages=c.cols)
    q = torch.full((T + 3, h, d), MARK, dtype=t, device=DEV)
    k = torch.full((T + 3, hkv, d), MARK, dtype=t, device=DEV)
    dev = lambda y: None if y is None else y.to(DEV)  # noqa: E731
    pl, ax = (None, None) if places is None else (on(places), on(axis))
    pools = run_append(cfg, c, qkv.to(DEV), dev(w), dev(f), cu, kv, q, k, pl, ax)
    q2, k2 = torch.full_like(q, MARK), torch.full_like(k, MARK)
    if axes:
        gdn.gdn_qk_norm_rope_axes(cfg, qkv.to(DEV), dev(w), dev(w), dev(f), pl, ax, on(cu), q2, k2)
    else:
        gdn.gdn_qk_norm_rope(cfg, qkv.to(DEV), dev(w), dev(w), dev(f), on(cu), ints(kv), q2, k2)
    assert torch.equal(q, q2) and torch.equal(k, k2) and (q[T:] == MARK).all()
    x = f64(qkv)[:T].reshape(T, h + 2 * hkv, d)
    part, w64 = x[:, h:h + hkv], None if w is None else f64(w)
    if axes:
        want, mag = cache8.norm_rope_axes(part, w64, places[:, :T], axis, f64(f), 1e-6, inter)
    elif rot or norm:
        want, mag = attention.norm_rope(part, w64, attention.positions(cu, kv), f64(f) if rot else None,
                                        1e-6, inter)
    else:
        want, mag = part, np.zeros_like(part)  # keys as they are: every code exactly
    check_append(c, pools, x, lens, kv, cu, want, mag, top_of(t))
    # the pages alone, and the same bits again
    again = run_append(cfg, c, qkv.to(DEV), dev(w), dev(f), cu, kv, None, None, pl, ax)
    for a, b in zip(pools, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [128, 256])
def test_append8_token_by_token(t, d):
    """A sequence that grows by one token a call, and by pieces, its tokens ever larger,
    ever smaller and by chance: the cache is the oracle's after every call."""
    h, hkv, page = 2, 2, 32
    rng = np.random.Generator(np.random.PCG64(8))
    for kind in ("grow", "shrink", "any"):
        c = Cache8([0], hkv, d, page, t, 12, extra_cols=3)
        c.table[0, :3] = [2, 0, 1]
        c.n_pages = 3
        shape = (3, hkv, page, d)
        c.k, c.v = (np.full(shape, 127, np.uint8) for _ in range(2))
        c.ks, c.vs = (np.full((3, hkv, page // 16), 251, np.uint8) for _ in range(2))
        kv = 0
        say(f"token by token {t} d={d} {kind}")
        for step in [1] * 18 + [3, 1, 5, 7, 1, 20, 1]:
            kv += step
            size = {"grow": 1.17 ** kv, "shrink": 0.8 ** kv, "any": 2.0 ** rng.integers(-9, 9)}[kind]
            x = normal(kv, step, (h + 2 * hkv) * d, dtype=t, scale=size)
            cfg = gdn.make_attn_config(step, 1, h, hkv, d, t, page_size=page, n_pages=3, max_pages=c.cols)
            pools = run_append(cfg, c, x.to(DEV), None, None, cu_of([step]), [kv], None, None)
            rows = f64(x).reshape(step, -1, d)
            check_append(c, pools, rows, [step], [kv], cu_of([step]), rows[:, h:h + hkv],
                         np.zeros((step, hkv, d)), top_of(t))
            c.k, c.v, c.ks, c.vs = (bytes_of(p) for p in pools)


@pytest.mark.parametrize("t", TYPES)
def test_append8_of_several_sequences_into_blocks_of_one_page(t):
    """Sequences may share a page, as long as each block is written by one of them."""
    h, hkv, d, page = 2, 2, 128, 64
    lens, kv = [5, 16, 1, 9], [16, 32, 40, 64]
    c = Cache8([64], hkv, d, page, t, 19)
    c.table = np.repeat(c.table[:1, :1], 4, 0)
    x = normal(20, sum(lens), (h + 2 * hkv) * d, dtype=t, scale=3.0)
    cfg = gdn.make_attn_config(sum(lens), 4, h, hkv, d, t, page_size=page, n_pages=c.n_pages, max_pages=1)
    say(f"append8, blocks of one page {t}")
    pools = run_append(cfg, c, x.to(DEV), None, None, cu_of(lens), kv, None, None)
    rows = f64(x).reshape(sum(lens), -1, d)
    check_append(c, pools, rows, lens, kv, cu_of(lens), rows[:, h:h + hkv],
                 np.zeros((sum(lens), hkv, d)), top_of(t))


@pytest.mark.parametrize("t", TYPES)
def test_append8_at_the_ends_of_the_types(t):
    """Zeros, the largest and the smallest numbers, NaN and infinities, single tokens and
    several, beside rows that a block had."""
    d, h, hkv, page = 128, 2, 2, 16
    big, small = torch.finfo(t).max, torch.finfo(t).smallest_normal
    for kv, new in (([5, 16, 1], [1, 1, 1]), ([9, 12, 16], [5, 3, 16])):
        T = sum(new)
        c = Cache8(kv, hkv, d, page, t, 14)
        x = normal(15, T, (h + 2 * hkv) * d, dtype=t)
        x[0] = 0
        x[1, ::3], x[1, 1::3] = big, -big
        x[-1, h * d:] = small * 0.25
        x[-1, -d:] = x[-1, -d:] * 0 + 1e-30
        x[0, h * d + 3], x[1, -1], x[2 % T, -d - 5] = float("nan"), float("inf"), float("-inf")
        say(f"append8, ends of the types {t} {new}")
        cfg = gdn.make_attn_config(T, 3, h, hkv, d, t, page_size=page, n_pages=c.n_pages, max_pages=c.cols)
        pools = run_append(cfg, c, x.to(DEV), None, None, cu_of(new), kv, None, None)
        rows = f64(x).reshape(T, -1, d)
        check_append(c, pools, rows, new, kv, cu_of(new), rows[:, h:h + hkv], np.zeros((T, hkv, d)), top_of(t))


@pytest.mark.parametrize("single", [True, False])
def test_append8_skips_rows_without_a_page(single):
    """Entries that name no page, columns past the table and negative positions."""
    t, d, page, hkv = torch.bfloat16, 128, 16, 1
    lens = [1, 1, 1, 1] if single else [2, 2, 2, 3]
    kv = np.array([2, 2, 50, 0 if single else 1], np.int32)  # 50: column 3 of 2; then below zero
    table = np.array([[-1, 0], [7, 0], [1, 2], [3, 3]], np.int32)  # 4 pages: 7 names none
    pools = [torch.full((4, hkv, page, d), 7, dtype=torch.uint8, device=DEV) for _ in range(2)]
    pools += [torch.full((4, hkv, 1), 9, dtype=torch.uint8, device=DEV) for _ in range(2)]
    say("append8 without pages")
    q = gdn.append_paged_kv(normal(1, sum(lens), 3 * d, dtype=t).to(DEV), 1, on(cu_of(lens)), on(kv),
                            on(table), *pools[:2], k_scales=pools[2], v_scales=pools[3])
    want = [] if single else [[3, 0, 0]]
    for p in pools[:2]:
        assert (p != 7).any(-1).nonzero().tolist() == want
    for p in pools[2:]:
        assert (p != 9).nonzero().tolist() == want
    assert q.isfinite().all()


def test_append8_with_malformed_batches_stays_inside():
    """Decreasing and oversized cu_seqlens, lengths and table entries of any kind: guards around
    q, k, the pools and the scales stay as they were."""
    t, h, hkv, d, T, n, page, pages = torch.bfloat16, 2, 2, 128, 40, 3, 16, 4
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, rot_dim=64, page_size=page, n_pages=pages, max_pages=2)
    x = normal(1, T, 6 * d).to(DEV)
    f, w = gdn.rope_inv_freq(64).to(DEV), torch.ones(d, device=DEV)
    bufs = [torch.full((T + 8, m, d), MARK, dtype=t, device=DEV) for m in (h, hkv)]
    pools = [torch.full((pages + 2, hkv, page, d), 5, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.full((pages + 32, hkv, 1), 5, dtype=torch.uint8, device=DEV) for _ in range(2)]
    table = ints([[0, 1], [-5, 9], [2_000_000_000, 3]])
    places, axis = on(places_of(T, 2, 1)), ints(np.arange(32) * 1000 - 9)
    for cu in ([0, 30, 10, 40], [0, -5, 90, 20], [7, 7, 60, 41]):
        for kv in ([32, 31, 2_000_000_000], [-4, -2_000_000_000, 5], [20, 1, 0]):
            for pos in ((None, None), (places, axis)):
                gdn.gdn_kv_append8(cfg, x, w, w, f, *pos, ints(cu), ints(kv), table, bufs[0][4:4 + T],
                                   bufs[1][4:4 + T], pools[0][1:1 + pages], pools[1][1:1 + pages],
                                   scales[0][16:16 + pages], scales[1][16:16 + pages])
            gdn.gdn_qk_norm_rope_axes(cfg, x, w, w, f, places, axis, ints(cu), bufs[0][4:4 + T],
                                      bufs[1][4:4 + T])
    for b in bufs:
        assert (b[:4] == MARK).all() and (b[4 + T:] == MARK).all()
    for p in pools:
        assert (p[0] == 5).all() and (p[-1] == 5).all()
    for s in scales:
        assert (s[:16] == 5).all() and (s[16 + pages:] == 5).all()


# ---------------------------------------------------------------- attention

PAGED = [
    # new tokens, tokens in all; h, hkv, d, page, shared
    ([1], [1], 1, 1, 128, 16, 0),
    ([1, 1, 1], [5, 129, 1000], 8, 2, 128, 16, 0),
    ([1, 1, 0, 1], [700, 0, 33, 17], 16, 2, 256, 32, 0),   # a row that sees no key
    ([4, 1, 9], [4, 40, 300], 8, 1, 128, 64, 0),
    ([8, 3], [5, 2], 4, 2, 128, 16, 0),                    # more tokens than keys
    ([16, 16], [2100, 16], 24, 2, 128, 128, 0),
    ([50, 1], [500, 260], 6, 2, 256, 256, 0),
    ([1] * 40, [150 + 7 * i for i in range(40)], 8, 2, 128, 16, 130),
    ([2, 1, 5, 1], [400, 513, 389, 700], 16, 2, 256, 64, 384),
    ([3, 3], [330, 200], 8, 1, 128, 16, 197),              # all after the prefix, to the token
    ([1, 6], [900, 500], 4, 1, 256, 32, 490),              # tokens reach into it: fewer pages
    ([1] * 300, [1 + i % 50 for i in range(300)], 2, 1, 128, 16, 0),
    ([1] * 20, [1100 + 9 * i for i in range(20)], 16, 2, 256, 16, 1000),  # prefix in parts
    ([60, 45], [700, 300], 8, 1, 128, 16, 0),              # many rows: tiles over the pages
    ([130, 0, 20], [130, 77, 1500], 8, 2, 256, 64, 0),
    ([90], [60], 8, 1, 128, 32, 0),
    ([300, 280], [400, 333], 2, 1, 128, 128, 64),
    ([1] * 100, [200 + i for i in range(100)], 4, 2, 128, 16, 150),   # more sequences than lanes
    ([1] * 280, [1 + 3 * i for i in range(280)], 16, 4, 128, 32, 0),  # a wave per joined row
    ([2] * 90, [500 - i for i in range(90)], 24, 2, 256, 16, 300),
    ([1, 2], [300, 40], 17, 1, 128, 16, 0),
    ([16 + i % 3 for i in range(70)], [600 + 7 * i for i in range(70)], 8, 1, 128, 64, 0),
    ([40] * 10, [900 + 31 * i for i in range(10)], 4, 1, 256, 32, 0),  # tiles with parts and without
    ([4] * 9, [700 + 90 * i for i in range(9)], 8, 1, 128, 16, 0),     # two row tiles per item
    ([8] * 9, [900 + 40 * i for i in range(9)], 8, 1, 128, 16, 400),   # four, behind a prefix
    ([8] * 9, [900 + 40 * i for i in range(9)], 16, 2, 256, 64, 400),  # and items of two row tiles
    ([1, 1], [90, 3], 2048, 1, 128, 16, 0),                            # very many heads
    # tiles with as many parts as their keys ask for: none to many, of more sequences than lanes too
    ([40, 0, 3, 64, 1], [2600, 900, 64, 300, 5], 8, 2, 128, 16, 0),
    ([70, 33], [3100, 40], 12, 2, 256, 32, 0),
    ([9 + i % 9 if i % 7 else 0 for i in range(70)], [20 + 45 * i for i in range(70)], 8, 1, 128, 64, 0),
    ([60 + i for i in range(12)], [2100 + i % 5 * 300 for i in range(12)], 8, 2, 128, 128, 0),
]


def shared_cols8(n, hkv, d, page):
    """Table columns with which n sequences of a batch are worth a pass of its own over a shared
    prefix as long as the table, at codes of one byte and at values of two."""
    return -(-(1 << 28) // (2 * n * hkv * d * page))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("new,full,h,hkv,d,page,shared", PAGED)
def test_paged8(t, new, full, h, hkv, d, page, shared):
    T, n = sum(new) + 2, len(new) + 1
    c = Cache8(list(full) + [0], hkv, d, page, t, 21, shared=shared)
    cu = cu_of(new, n)
    q = normal(1, T, h, d, dtype=t)
    q[int(cu[-1]):] = float("nan")
    say(f"paged8 {t} n={len(new)} tokens={sum(new)} keys={sum(full)} h={h} hkv={hkv} d={d} "
        f"page={page} shared={shared}")
    pools = c.on()
    for cols in [c.cols] + ([shared_cols8(n, hkv, d, page)] if shared else []):
        cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=c.n_pages,
                                   max_pages=cols, shared_max=cols * page if shared else 0)
        o = torch.full((T, h, d), MARK, dtype=t, device=DEV)
        sh = ints([shared]) if shared else None
        args = (q.to(DEV), *pools, on(cu), ints(c.lens), on(widened(c.table, cols)))
        gdn.gdn_attn_paged8(cfg, *args, sh, o, workspace(cfg))
        worst = 0.0
        for s in range(len(new)):
            a = slice(cu[s], cu[s + 1])
            k, v = c.rows(s)
            worst = max(worst, check_attention(o[a], f64(q[a]), k, v, d ** -0.5, t))
        say(f"  off / bound {worst:.3f}")
        assert (o[sum(new):] == MARK).all()
    # the same bits again, with another workspace's content
    o2 = torch.full_like(o, MARK)
    gdn.gdn_attn_paged8(cfg, *args, sh, o2, torch.zeros_like(workspace(cfg)))
    assert torch.equal(o, o2)


LONG = [
    # new tokens, older keys of each; h, hkv, d, page; every how many rows
    ([2300], 333, 8, 2, 128, 64, 301), ([4096], 0, 32, 8, 128, 256, 701), ([1100], 900, 16, 2, 256, 16, 211),
    ([60, 3, 45], 900, 8, 1, 256, 16, 7), ([3000, 1700], 40, 16, 4, 128, 32, 401),
    ([i % 60 for i in range(100)], 30, 8, 1, 128, 16, 31), ([i % 40 for i in range(100)], 10, 16, 2, 256, 128, 31),
    ([4 + i % 12 for i in range(300)], 25, 8, 1, 128, 16, 61),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lens,past,h,hkv,d,page,step", LONG)
def test_paged8_of_prompts_at_sampled_rows(t, lens, past, h, hkv, d, page, step):
    """Tiles of every kind (four and eight waves, keys in parts, every search)."""
    full = [x + past for x in lens]
    T, n, cu = sum(lens), len(lens), cu_of(lens)
    c = Cache8(full, hkv, d, page, t, 40, extra_cols=0)
    q = normal(1, T, h, d, dtype=t)
    say(f"prompts over 8-bit pages {t} n={n} T={T} past={past} h={h} hkv={hkv} d={d}")
    kp, vp, ks, vs = c.on()
    args = (q.to(DEV), kp, vp, on(cu), ints(full), on(c.table))
    o = gdn.paged_attention(*args, k_scales=ks, v_scales=vs)
    assert o.isfinite().all()
    rows_of = functools.lru_cache(None)(c.rows)
    for at in sorted({*range(0, T, step), *(int(x) - 1 for x in cu[1:])} - {-1}):
        s = int(np.searchsorted(cu[1:], at, side="right"))
        seen = past + at - int(cu[s]) + 1
        k, v = rows_of(s)
        check_attention(o[at:at + 1], f64(q[at:at + 1]), k[:seen], v[:seen], d ** -0.5, t)
    assert torch.equal(o, gdn.paged_attention(*args, k_scales=ks, v_scales=vs))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("new,full,h,hkv,d", [([1, 1, 1], [70, 900, 3000], 16, 2, 128),
                                              ([5, 2], [600, 77], 8, 2, 256),
                                              ([200, 130], [700, 900], 8, 2, 128),
                                              ([300], [2000], 16, 2, 256)])
def test_paged8_is_the_16_bit_call_on_the_caches_numbers(t, new, full, h, hkv, d):
    """Codes turned into the 16-bit type by torch, and the 16-bit call on them: the same scores
    and weights in another order at most, so within two of the output's steps."""
    c = Cache8(full, hkv, d, 32, t, 23)
    q = normal(1, sum(new), h, d, dtype=t).to(DEV)
    kp, vp, ks, vs = c.on()
    say(f"8 and 16 bits {t} {new} d={d}")
    batch = (on(cu_of(new)), ints(full), on(c.table))
    o = gdn.paged_attention(q, kp, vp, *batch, k_scales=ks, v_scales=vs)
    wide = [(x.float() * s.float().repeat_interleave(16, 2)[..., None]).to(t) for x, s in ((kp, ks), (vp, vs))]
    o16 = gdn.paged_attention(q, *wide, *batch)
    step = torch.finfo(t).eps * o16.float().abs() + 2 * torch.finfo(t).eps * float(o16.float().abs().max()) * 2 ** -4
    assert ((o.float() - o16.float()).abs() <= 2 * step).all()


@pytest.mark.parametrize("new,full,h,hkv,d,page,shared", [
    ([1, 1], [9000, 700], 8, 2, 128, 16, 0),                 # keys in parts, four waves per row
    ([1] * 300, [100 + 3 * i for i in range(300)], 16, 4, 128, 32, 0),  # and one wave per row
    ([1, 2, 1], [900, 950, 1200], 16, 2, 256, 16, 700),      # beside a shared prefix
    ([200, 40], [500, 40], 8, 2, 128, 16, 0),                # tiles over the pages
    ([140], [4000], 4, 2, 256, 64, 0),                       # with their keys in parts
])
def test_paged8_keeps_what_is_not_finite_in_its_rows(new, full, h, hkv, d, page, shared):
    """NaN in a query row, in a code, or in a block's scale comes out of the rows that read it and
    of no other sequence's."""
    t = torch.bfloat16
    for code in (True, False):
        c = Cache8(full, hkv, d, page, t, 3, shared)
        q = normal(1, sum(new), h, d, dtype=t)
        q[0, 0] = float("nan")
        last = len(new) - 1
        at = full[last] - 1 - new[last] // 2  # the last sequence's, behind the prefix
        if code:
            c.v[c.table[last, at // page], :, at % page] = 127
        else:
            c.vs[c.table[last, at // page], :, at % page // 16] = 255
        kp, vp, ks, vs = c.on()
        cu = cu_of(new)
        say(f"paged8, values that are not finite {new[:4]} {full[:4]} d={d} shared={shared}")
        table = widened(c.table, shared_cols8(len(new), hkv, d, page)) if shared else c.table
        o = gdn.paged_attention(q.to(DEV), kp, vp, on(cu), ints(full), on(table),
                                ints([shared]) if shared else None, k_scales=ks, v_scales=vs)
        assert o[0, 0].isnan().all()
        b = int(cu[last]) if last else 0
        if last:
            assert o[:b].flatten(0, 1)[1:].isfinite().all()
        first = at if code else at // 16 * 16
        reads = full[last] - new[last] + np.arange(new[last]) >= first
        assert not o[b:][torch.from_numpy(reads).to(DEV)].isfinite().any()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("new,full", [([1], [300]), ([40], [300]), ([40], [3000])])
def test_paged8_of_scales_at_their_ends(t, new, full):
    """Blocks of tiny, of huge and of zero numbers side by side: what the 16-bit type holds of
    them is what counts."""
    h, hkv, d, page = 8, 1, 128, 32
    c = Cache8(full, hkv, d, page, t, 25)
    rng = np.random.Generator(np.random.PCG64(4))
    n = full[0] // 16
    lo, hi = (110, 121) if t == torch.float16 else (15, 150)
    for p in range(n):
        page_, b = c.table[0, p * 16 // page], p * 16 % page // 16
        c.ks[page_, :, b] = 105 if p % 3 else 111
        c.vs[page_, :, b] = rng.integers(lo, hi)
        if p % 7 == 0:
            c.v[page_, :, b * 16:b * 16 + 16] = 128  # -0
    q = normal(2, new[0], h, d, dtype=t)
    say(f"paged8, scales {t} {new} {full}")
    kp, vp, ks, vs = c.on()
    o = gdn.paged_attention(q.to(DEV), kp, vp, on(cu_of(new)), ints(full), on(c.table), k_scales=ks,
                            v_scales=vs)
    k, v = (f64(torch.from_numpy(x).to(t)) for x in c.rows(0))
    check_attention(o, f64(q), k, v, d ** -0.5, t)


@pytest.mark.parametrize("d,hkv", [(128, 8), (256, 4)])
def test_paged8_of_more_keys_than_the_caches_hold(d, hkv):
    """132000 keys of 2048 bytes, read past the caches: a streamed row and tiles in parts."""
    t, h, T, lens = torch.bfloat16, 4 * hkv, 20, [132000, 300]
    c = Cache8(lens, hkv, d, 256, t, 17)
    kp, vp, ks, vs = c.on()
    q = normal(5, T + 1, h, d, dtype=t)
    for new in ([1, 1], [T, 1]):
        say(f"more 8-bit keys than the caches hold d={d} new={new}")
        cu = cu_of(new)
        o = gdn.paged_attention(q[:sum(new)].to(DEV), kp, vp, on(cu), ints(lens), on(c.table), k_scales=ks,
                                v_scales=vs)
        for s in range(2):
            rows = [int(cu[s]), int(cu[s + 1]) - 1]
            k, v = c.rows(s)
            for r in set(rows):
                seen = lens[s] - (int(cu[s + 1]) - 1 - r)
                check_attention(o[r:r + 1], f64(q[r:r + 1]), k[:seen], v[:seen], d ** -0.5, t)


def test_paged8_indexes_that_name_nothing_stay_inside():
    """Lengths past the table, entries past the pool and a decreasing cu_seqlens give some
    values, and write only rows of o."""
    t, h, hkv, d, page = torch.bfloat16, 4, 1, 128, 16
    n, T, pages = 5, 12, 3
    c = Cache8([page * pages], hkv, d, page, t, 2, spare=0)
    pools = c.on()
    table = np.array([[0, 1], [-5, 9], [2_000_000_000, 1], [1, -2_000_000_000], [2, 2]], np.int32)
    buf = torch.full((T + 8, h, d), MARK, dtype=t, device=DEV)
    q, sh = normal(3, T, h, d).to(DEV), ints([1 << 30])
    for cols in (2, shared_cols8(n, hkv, d, page)):
        cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=pages, max_pages=cols,
                                   shared_max=64 if cols == 2 else 1 << 30)
        wide = on(widened(table, cols))
        for cu in ([0, 2, 3, 9, 10, 12], [0, 9, 4, 4, 20, 11], [5, 3, -7, 12, 1, 40]):
            for kv in ([32, 31, 20, 2_000_000_000, 0], [-4, 1000, 32, 32, 32]):
                gdn.gdn_attn_paged8(cfg, q, *pools, ints(cu), ints(kv), wide, sh, buf[4:4 + T], workspace(cfg))
                assert (buf[:4] == MARK).all() and (buf[4 + T:] == MARK).all()


@pytest.mark.parametrize("d", [128, 256])
def test_paged8_indexes_that_name_nothing_stay_inside_of_tiles_in_parts(d):
    t, h, hkv, page, n, T, pages, cols = torch.bfloat16, 8, 1, 16, 3, 150, 3, 60
    c = Cache8([page * pages], hkv, d, page, t, 2, spare=0)
    pools = c.on()
    table = np.arange(n * cols, dtype=np.int32).reshape(n, cols) % 7 - 2
    table[1, ::5], table[2, ::3] = 2_000_000_000, -2_000_000_000
    buf = torch.full((T + 8, h, d), MARK, dtype=t, device=DEV)
    q = normal(3, T, h, d).to(DEV)
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=pages, max_pages=cols)
    size = gdn.gdn_attn_paged8_workspace_size(cfg)
    assert size > 256  # parts
    for cu in ([0, 70, 80, 150], [0, 150, 0, 150], [0, 2_000_000_000, -5, 150], [7, 150, 149, 60]):
        for kv in ([960, 900, 3], [-4, 2_000_000_000, 500], [2_000_000_000] * 3):
            ws = torch.full((size + 512,), 0x55, dtype=torch.uint8, device=DEV)
            gdn.gdn_attn_paged8(cfg, q, *pools, ints(cu), ints(kv), ints(table), None, buf[4:4 + T],
                                ws[256:256 + size])
            assert (buf[:4] == MARK).all() and (buf[4 + T:] == MARK).all()
            assert (ws[:256] == 0x55).all() and (ws[256 + size:] == 0x55).all()


@pytest.mark.parametrize("d", [128, 256])
def test_batches_without_tokens_write_nothing(d):
    t, h, hkv, page, n, T = torch.float16, 4, 2, 16, 3, 9
    pools = [torch.full((5, hkv, page, d), 7, dtype=torch.uint8, device=DEV) for _ in range(2)]
    pools += [torch.full((5, hkv, 1), 7, dtype=torch.uint8, device=DEV) for _ in range(2)]
    cu, kv, table = ints([0] * (n + 1)), ints([20] * n), ints(np.zeros((n, 2)))
    x = normal(1, T, (h + 2 * hkv) * d, dtype=t).to(DEV)
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, rot_dim=32, page_size=page, n_pages=5, max_pages=2)
    q, o = (torch.full((T, h, d), MARK, dtype=t, device=DEV) for _ in range(2))
    k = torch.full((T, hkv, d), MARK, dtype=t, device=DEV)
    f, places, axis = gdn.rope_inv_freq(32).to(DEV), on(places_of(T, 2, 1)), ints([0] * 16)
    gdn.gdn_qk_norm_rope_axes(cfg, x, None, None, f, places, axis, cu, q, k)
    gdn.gdn_kv_append8(cfg, x, None, None, f, None, None, cu, kv, table, q, k, *pools)
    gdn.gdn_attn_paged8(cfg, q, *pools, cu, kv, table, None, o, workspace(cfg))
    for y in (q, k, o):
        assert (y == MARK).all()
    for y in pools:
        assert (y == 7).all()


# ---------------------------------------------------------------- large

def test_both_capacity_limits_with_sequences_at_the_end():
    """t_max = 2^24 rows and n_max = 16384 sequences, the checked ones the last two: norm and
    rotation by axes and the append; then a decode step of 16384 sequences."""
    t, d, h, hkv, page = torch.bfloat16, 128, 1, 1, 256
    T, n = gdn.GDN_T_MAX_LIMIT, gdn.GDN_N_MAX_LIMIT
    tail = [70, 3]
    cu = np.zeros(n + 1, np.int64)
    cu[:n - 1] = np.linspace(0, T - sum(tail), n - 1).astype(np.int64)
    cu[n - 1:] = T - tail[1], T
    say(f"capacity limits: {T} rows, {n} sequences")
    x = torch.zeros(T, 3 * d, dtype=t, device=DEV)
    rows = normal(1, sum(tail), 3 * d, dtype=t)
    x[T - sum(tail):] = rows.to(DEV)
    f = gdn.rope_inv_freq(d).to(DEV)
    places = torch.zeros(3, T, dtype=torch.int32, device=DEV)
    last = places_of(sum(tail), 3, 2)
    places[:, T - sum(tail):] = on(last)
    axis = gdn.rope_pair_axis([22, 21, 21], True)
    cud = on(cu.astype(np.int32))
    q, k = gdn.qk_norm_rope(x, h, hkv, cud, inv_freq=f, positions=places, pair_axis=axis.to(DEV))
    xs = f64(rows).reshape(-1, 3, d)
    for got, part in ((q, xs[:, :1]), (k, xs[:, 1:2])):
        want, mag = cache8.norm_rope_axes(part, None, last, axis.numpy(), f64(f), 1e-6)
        check_norm_rope(got[-sum(tail):], want, mag, t)
        assert not got[:T - sum(tail)].any()
    del q, k, places
    # only the last two sequences have pages
    c = Cache8([0, 0], hkv, d, page, t, 5, extra_cols=1)
    c.n_pages = 2
    c.k, c.v = (np.full((2, hkv, page, d), 3, np.uint8) for _ in range(2))
    c.ks, c.vs = (np.full((2, hkv, page // 16), 120, np.uint8) for _ in range(2))
    table = np.full((n, 1), -1, np.int32)
    table[n - 2:, 0] = 1, 0
    kv = np.diff(cu).astype(np.int32)
    kp, vp, ks, vs = c.on()
    gdn.append_paged_kv(x, h, cud, on(kv), on(table), kp, vp, k_scales=ks, v_scales=vs)
    c.table = table[n - 2:]
    check_append(c, (kp, vp, ks, vs), xs, tail, tail, cu_of(tail), xs[:, 1:2], np.zeros_like(xs[:, 1:2]), top_of(t))
    del x
    qq = torch.zeros(n, h, d, dtype=t, device=DEV)
    qq[n - 2:] = normal(6, 2, h, d, dtype=t).to(DEV)
    table[:n - 2] = 0
    kv[:n - 2] = 1
    o = gdn.paged_attention(qq, kp, vp, ints(np.arange(n + 1)), on(kv), on(table), k_scales=ks, v_scales=vs)
    c.k, c.v, c.ks, c.vs = (bytes_of(y) for y in (kp, vp, ks, vs))
    c.lens = tail
    first = torch.from_numpy(c.rows(1)[1][0]).to(t).to(DEV)
    assert torch.equal(o[:n - 2], first.expand(n - 2, 1, d))
    for i in range(2):
        check_attention(o[n - 2 + i:n - 1 + i], f64(qq[n - 2 + i:n - 1 + i]), *c.rows(i), d ** -0.5, t)
    torch.cuda.empty_cache()


def test_offsets_past_32_bits_in_a_large_pool():
    """Pages whose byte offsets pass 2^32, written by append and read by attention."""
    t, h, hkv, d, page = torch.bfloat16, 4, 2, 256, 256
    pages = 33000  # 33000 * 2 * 256 * 256 bytes: 4.3e9
    kp, vp = (torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(pages, hkv, page // 16, dtype=torch.uint8, device=DEV) for _ in range(2))
    n = 300
    table = np.array([[pages - 1, 32900]], np.int32)
    x = normal(5, n, (h + 2 * hkv) * d, dtype=t)
    kv, cu = ints([n]), on(cu_of([n]))
    say("offsets past 32 bits")
    q = gdn.append_paged_kv(x.to(DEV), h, cu, kv, on(table), kp, vp, k_scales=ks, v_scales=vs)
    assert not kp[:32900].any() and not vp[32901:-1].any() and not ks[32901:-1].any()
    c = Cache8([n], hkv, d, page, t, 1, extra_cols=0)
    c.k, c.v, c.ks, c.vs = (bytes_of(torch.stack([y[pages - 1], y[32900]])) for y in (kp, vp, ks, vs))
    c.table = np.array([[0, 1]], np.int32)
    xs = f64(x).reshape(n, -1, d)
    for name, rows in (("k", xs[:, h:h + hkv]), ("v", xs[:, h + hkv:])):
        codes, scales = np.zeros_like(c.k), np.zeros_like(c.ks)
        cache8.append(codes, scales, c.table[0], 0, rows, top_of(t))
        assert np.array_equal(getattr(c, name), codes) and np.array_equal(getattr(c, name + "s"), scales)
    for new in (1, 40):
        o = gdn.paged_attention(q[-new:].contiguous(), kp, vp, on(cu_of([new])), kv, on(table), k_scales=ks,
                                v_scales=vs)
        check_attention(o, f64(q[-new:]), *c.rows(0), d ** -0.5, t)
    del kp, vp
    torch.cuda.empty_cache()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,rot,axes", [(128, 128, 3), (256, 64, 0)])
def test_a_large_append_equals_its_blocks(t, d, rot, axes):
    """40000 tokens of uneven sequences in one call against pieces of whole blocks."""
    h, hkv, page = 2, 2, 64
    lens = [20007, 1, 16, 19976]
    T = sum(lens)
    x = torch.randn(T, (h + 2 * hkv) * d, device=DEV).to(t)
    f = gdn.rope_inv_freq(rot).to(DEV)
    pages = sum(-(-n // page) for n in lens)
    table = np.zeros((4, -(-max(lens) // page)), np.int32)
    at = 0
    for i, n in enumerate(lens):
        table[i, :-(-n // page)] = range(at, at + -(-n // page))
        at += -(-n // page)
    pools = [[torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device=DEV) for _ in range(2)] +
             [torch.zeros(pages, hkv, page // 16, dtype=torch.uint8, device=DEV) for _ in range(2)]
             for _ in range(2)]
    places = on(places_of(T, axes, 3)) if axes else None
    axis = (torch.arange(rot // 2) % axes).int().to(DEV) if axes else None
    say(f"large append8 {t} T={T} d={d}")

    def append(a, b, seqs, ends, p):
        cu = cu_of([max(min(b, int(c1)) - max(a, int(c0)), 0) for c0, c1 in seqs])
        return gdn.append_paged_kv(x[a:b], h, on(cu), ints(ends), on(table), *p[:2], inv_freq=f,
                                   k_scales=p[2], v_scales=p[3], output_k=True, pair_axis=axis,
                                   positions=places[:, a:b].contiguous() if axes else None)

    cu = cu_of(lens)
    seqs = list(zip(cu[:-1], cu[1:]))
    q, k = append(0, T, seqs, lens, pools[0])
    parts, a = [], 0
    for b in (16 * 400, 16 * 401, 20007, 20008 + 16 + 16 * 9, T):  # whole blocks of each sequence
        ends = [max(min(b, int(c1)) - int(c0), 0) for c0, c1 in seqs]
        parts.append(append(a, b, seqs, ends, pools[1]))
        a = b
    assert torch.equal(q, torch.cat([y[0] for y in parts])) and torch.equal(k, torch.cat([y[1] for y in parts]))
    assert all(torch.equal(y, z) for y, z in zip(*pools))


# ---------------------------------------------------------------- as they are used together

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,page,rot,inter", [(128, 16, 128, False), (256, 64, 64, True)])
def test_prompt_then_steps(t, d, page, rot, inter):
    """Two prompts of text and an image that begin alike: norm, rotation by three axes and append
    to an 8-bit cache, attention over it, then decode and verify steps with the shared pages read
    once. The cache against the oracle's at every step, outputs against the oracle on the numbers
    that the cache then holds."""
    h, hkv, common = 8, 2, 70
    lens = [90, 75]
    steps = [[1, 1], [3, 0], [2, 4], [1, 1]]
    total = [lens[i] + sum(s[i] for s in steps) for i in range(2)]
    sp = common // page
    need = [-(-x // page) for x in total]
    pages = sp + sum(x - sp for x in need)
    c = Cache8([0, 0], hkv, d, page, t, 1)
    c.table = np.full((2, max(need)), -1, np.int32)
    c.table[0, :need[0]] = range(need[0])
    c.table[1, :need[1]] = list(range(sp)) + list(range(need[0], pages))
    c.n_pages = pages
    c.k, c.v = (np.full((pages, hkv, page, d), 127, np.uint8) for _ in range(2))
    c.ks, c.vs = (np.full((pages, hkv, page // 16), 255, np.uint8) for _ in range(2))
    w = [normal(i, d, dtype=torch.float32, scale=0.3).add(1.0).to(DEV) for i in (1, 2)]
    f = gdn.rope_inv_freq(rot, 1e6).to(DEV)
    axis = gdn.rope_pair_axis([rot // 4, rot // 8, rot // 8], interleaved=inter)
    width = (h + 2 * hkv) * d
    same = normal(40, common, width, dtype=t)

    def places(first, n):
        """Text, but for an image of 6 by 7 that starts at position 20."""
        out = []
        for p in range(first, first + n):
            if 20 <= p < 62:
                out.append((20, 20 + (p - 20) // 7, 20 + (p - 20) % 7))
            else:
                out.append((p if p < 20 else p - 62 + 27,) * 3)
        return np.array(out, np.int32).reshape(n, 3).T

    def step(x, new, kv, shared):
        """One call of each; the sequences that begin alike write the shared pages once."""
        cu = cu_of(new)
        pos = np.concatenate([places(kv[s] - new[s], new[s]) for s in range(2)], 1)
        pools = c.on()
        q, k = gdn.append_paged_kv(x.to(DEV), h, on(cu), ints(kv), on(c.table), *pools[:2], *w, f,
                                   interleaved=inter, output_k=True, k_scales=pools[2],
                                   v_scales=pools[3], positions=on(pos), pair_axis=axis.to(DEV))
        xs = f64(x).reshape(-1, h + 2 * hkv, d)
        args = (pos, axis.numpy(), f64(f), 1e-6, inter)
        want, mag = cache8.norm_rope_axes(xs[:, :h], f64(w[0]), *args)
        check_norm_rope(q, want, mag, t)
        want, mag = cache8.norm_rope_axes(xs[:, h:h + hkv], f64(w[1]), *args)
        check_norm_rope(k, want, mag, t)
        check_append(c, pools, xs, new, kv, cu, want, mag, top_of(t))
        c.k, c.v, c.ks, c.vs = (bytes_of(p) for p in pools)
        table = widened(c.table, shared_cols8(2, hkv, d, page)) if shared else c.table
        o = gdn.paged_attention(q, *pools[:2], on(cu), ints(kv), on(table),
                                ints([common]) if shared else None, k_scales=pools[2], v_scales=pools[3])
        for s in range(2):
            a = slice(cu[s], cu[s + 1])
            check_attention(o[a], f64(q[a]), *c.rows(s, kv[s]), d ** -0.5, t)

    # the second prompt finds the first's whole pages there
    step(torch.cat([same, normal(41, lens[0] - common, width, dtype=t)]), [lens[0], 0], [lens[0], 0], False)
    tail = torch.cat([same[sp * page:], normal(42, lens[1] - common, width, dtype=t)])
    step(tail, [0, len(tail)], lens, False)
    kv = list(lens)
    for i, new in enumerate(steps):
        kv = [kv[s] + new[s] for s in range(2)]
        step(normal(50 + i, sum(new), width, dtype=t), new, kv, True)


def test_a_captured_decode_step_replays_with_other_lengths():
    """append + attention over an 8-bit cache in one graph: lengths, tables, positions and the
    shared length are read on the device, so one capture serves every step."""
    t, h, hkv, d, page, n = torch.bfloat16, 8, 2, 128, 16, 6
    rng = np.random.Generator(np.random.PCG64(3))
    cols, most = 40, shared_cols8(n, hkv, d, page)
    pages = n * cols
    c = Cache8([pages * page], hkv, d, page, t, 4, spare=0)
    table = on(widened(rng.permutation(pages).reshape(n, cols).astype(np.int32), most))
    pools = c.on()
    cfg = gdn.make_attn_config(2 * n, n, h, hkv, d, t, rot_dim=128, page_size=page, n_pages=pages,
                               max_pages=most, shared_max=most * page)
    x = torch.zeros(2 * n, (h + 2 * hkv) * d, dtype=t, device=DEV)
    cu, kv = on(cu_of([1] * n)), ints([5] * n)
    sh, places = ints([0]), ints(np.zeros((3, 2 * n)))
    axis = gdn.rope_pair_axis([24, 20, 20], device=DEV)
    f, w = gdn.rope_inv_freq(128).to(DEV), torch.ones(d, device=DEV)
    q, o = (torch.zeros(2 * n, h, d, dtype=t, device=DEV) for _ in range(2))

    def step(q, o, pools, ws):
        gdn.gdn_kv_append8(cfg, x, w, w, f, places, axis, cu, kv, table, q, None, *pools)
        gdn.gdn_attn_paged8(cfg, q, *pools, cu, kv, table, sh, o, ws)

    ws = workspace(cfg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q, o, pools, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q, o, pools, ws)
    for i in range(6):
        new = [1] * n if i % 2 == 0 else [0, 2, 3, 1, 4, 2]
        cu.copy_(on(cu_of(new)))
        kv.copy_(ints(rng.integers(200, cols * page, n)))
        table[:, :12] = table[0, :12] if i in (2, 3) else table[:, :12]
        sh.fill_(170 if i in (2, 3) else 0)
        places.copy_(on(places_of(2 * n, 3, i)))
        x.copy_(normal(60 + i, *x.shape))
        other = [p.view(torch.uint8).clone() for p in pools]
        q2, o2 = torch.zeros_like(q), torch.zeros_like(o)
        o.zero_(), q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        step(q2, o2, other, workspace(cfg))
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(q, q2), i
        assert all(torch.equal(a.view(torch.uint8), b) for a, b in zip(pools, other)), i


@pytest.mark.parametrize("d", [128, 256])
def test_captured_tiles_in_parts_replay_with_other_lengths(d):
    """How many parts a tile's keys are cut in goes by lengths on the device: one capture
    serves uneven, empty and short sequences, and a workspace of any content."""
    t, h, hkv, page, n, T, cols = torch.bfloat16, 8, 2, 32, 5, 120, 90
    rng = np.random.Generator(np.random.PCG64(9))
    c = Cache8([cols * page] * n, hkv, d, page, t, 6, extra_cols=0)
    pools, table = c.on(), on(c.table)
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=c.n_pages, max_pages=cols)
    q, o = (torch.zeros(T, h, d, dtype=t, device=DEV) for _ in range(2))
    cu, kv = on(cu_of([24] * n)), ints([100] * n)
    ws = workspace(cfg)
    args = (cfg, q, *pools, cu, kv, table, None)
    gdn.gdn_attn_paged8(*args, o, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_attn_paged8(*args, o, ws)
    for i, (new, full) in enumerate([([24] * n, [2880] * n), ([100, 0, 3, 16, 1], [2880, 7, 900, 16, 300]),
                                     ([1, 1, 1, 1, 80], [5, 2880, 600, 0, 2500]), ([0] * n, [0] * n),
                                     ([17, 40, 16, 20, 27], rng.integers(30, 2880, n))]):
        cu.copy_(on(cu_of(new)))
        kv.copy_(ints(full))
        q.copy_(normal(70 + i, T, h, d, dtype=t))
        say(f"captured tiles in parts d={d} {new}")
        o.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        for s in range(n):
            at = slice(sum(new[:s]), sum(new[:s + 1]))
            k, v = c.rows(s, int(full[s]))
            check_attention(o[at], f64(q[at]), k, v, d ** -0.5, t)
        assert (o[sum(new):] == MARK).all()
        o2 = torch.full_like(o, MARK)
        gdn.gdn_attn_paged8(*args, o2, torch.zeros_like(ws))
        assert torch.equal(o, o2)


@pytest.mark.parametrize("d", [128, 256])
def test_two_graphs_that_share_a_workspace(d):
    """A prompt over 8-bit pages, whole and with its keys in parts, and a decode step, captured
    apart with one workspace and replayed in turn: nothing in it outlives a call."""
    t, h, hkv, page = torch.bfloat16, 8, 2, 32
    c = Cache8([1500, 260], hkv, d, page, t, 90)
    pools, table = c.on(), on(c.table)
    kv = ints(c.lens)
    q = normal(91, 1300, h, d, dtype=t).to(DEV)
    news = [[100, 200], [1100, 200], [1, 1]]
    cus = [on(cu_of(x)) for x in news]
    cfgs = [gdn.make_attn_config(sum(x), 2, h, hkv, d, t, page_size=page, n_pages=c.n_pages, max_pages=c.cols)
            for x in news]
    calls = [lambda o, ws, i=i: gdn.gdn_attn_paged8(cfgs[i], q[:sum(news[i])], *pools, cus[i], kv, table, None,
                                                    o[:sum(news[i])], ws) for i in range(3)]
    want = []
    for cfg, call in zip(cfgs, calls):
        want.append(torch.zeros_like(q))
        call(want[-1], workspace(cfg))
    ws = torch.empty(max(gdn.gdn_attn_paged8_workspace_size(x) for x in cfgs), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        outs.append(torch.zeros_like(q))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(outs[-1], ws)
    for i in range(4):
        for j in (0, 2, 1) if i % 2 else (1, 0, 2):
            outs[j].zero_()
            graphs[j].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), i


def test_two_streams_with_their_own_workspaces():
    t, h, hkv, d, page = torch.float16, 8, 1, 128, 16
    runs = []
    for i in range(2):
        c = Cache8([3000 + 500 * i, 40], hkv, d, page, t, 70 + i)
        q = normal(80 + i, 2, h, d, dtype=t).to(DEV)
        kp, vp, ks, vs = c.on()
        runs.append(((q, kp, vp, on(cu_of([1, 1])), ints(c.lens), on(c.table)), dict(k_scales=ks, v_scales=vs)))
    alone = [gdn.paged_attention(*a, **k) for a, k in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        outs = []
        for s, (a, k) in zip(streams, runs):
            with torch.cuda.stream(s):
                outs.append(gdn.paged_attention(*a, **k))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
