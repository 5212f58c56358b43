"""GPU parity of the softmax-attention operators (norm + rotation, append to the
paged cache, prefill attention, paged attention) against the fp64 CPU oracle,
through the C ABI. The bounds are derived in attn_helpers.py."""

import numpy as np
import pytest
import torch

import chunked_gated_delta_rule_amd as gdn
from attn_helpers import (DEV, TYPES, Cache, check_attention, check_norm_rope, cu_of, f64, normal,
                          on, shared_cols, widened)
from oracle import attention

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
    return torch.full((gdn.gdn_attn_workspace_size(cfg),), 0xff, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------- norm + rotation, append

ROTS = [(128, 128, False), (128, 128, True), (128, 0, False), (128, 2, False), (128, 66, False),
        (128, 64, True), (256, 64, False), (256, 256, False), (256, 250, False), (256, 10, True)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,rot,inter", ROTS)
def test_norm_rope(t, d, rot, inter):
    lens, h, hkv, spare = [3, 0, 1, 17], 6, 2, 4
    T = sum(lens)
    cu = cu_of(lens, len(lens) + 1)
    kv = np.array([3, 5, 2_000_000_000, 40, 9], np.int32)
    qkv = normal(d + rot, T + spare, (h + 2 * hkv) * d, dtype=t)
    qw, kw = normal(1, d, dtype=torch.float32), normal(2, d, dtype=torch.float32)
    f = gdn.rope_inv_freq(rot, 10000.0) if rot else None
    say(f"norm_rope {t} d={d} rot={rot} inter={inter}")
    cfg = gdn.make_attn_config(T + spare, len(lens) + 1, h, hkv, d, t, rot_dim=rot,
                               rot_interleaved=inter, rot_scale=1.25, eps=1e-5)
    q = torch.full((T + spare, h, d), MARK, dtype=t, device=DEV)
    k = torch.full((T + spare, hkv, d), MARK, dtype=t, device=DEV)
    gdn.gdn_qk_norm_rope(cfg, qkv.to(DEV), qw.to(DEV), kw.to(DEV), None if f is None else f.to(DEV),
                         on(cu), on(kv), q, k)
    x = f64(qkv)[:T].reshape(T, h + 2 * hkv, d)
    pos = attention.positions(cu, kv)
    for got, part, w in ((q, x[:, :h], qw), (k, x[:, h:h + hkv], kw)):
        want, mag = attention.norm_rope(part, f64(w), pos, None if f is None else f64(f), 1e-5,
                                        inter, 1.25)
        check_norm_rope(got[:T], want, mag, t)
        assert (got[T:] == MARK).all()  # rows behind the last sequence


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("T,d,rot,inter", [(5000, 128, 128, False), (10001, 128, 34, False),
                                           (9000, 256, 64, True)])
def test_norm_rope_and_append_of_many_tokens(t, T, d, rot, inter):
    """Several tokens per work-group, sequences that begin and end inside one."""
    h, hkv, page = 2, 1, 32
    lens = [7, 1, 0, 2, 1500, 3, 1]
    lens.append(T - sum(lens))
    n = len(lens)
    kv = [x + 11 * i for i, x in enumerate(lens)]
    cu = cu_of(lens)
    qkv = normal(30, T, 4 * d, dtype=t).to(DEV)
    w = normal(31, d, dtype=torch.float32).to(DEV)
    f = gdn.rope_inv_freq(rot).to(DEV)
    need = [-(-x // page) for x in kv]
    cols = max(need)
    table = np.zeros((n, cols), np.int32)
    at = 0
    for i, u in enumerate(need):
        table[i, :u] = range(at, at + u)
        at += u
    kp = torch.full((at, hkv, page, d), MARK, dtype=t, device=DEV)
    vp = kp.clone()
    say(f"norm_rope / append {t} T={T} d={d} rot={rot}")
    q, k = gdn.append_paged_kv(qkv, h, on(cu), on(np.array(kv, np.int32)), on(table), kp, vp, w,
                               None, f, interleaved=inter, output_k=True)
    x = f64(qkv).reshape(T, 4, d)
    pos = attention.positions(cu, kv)
    for got, part, wt in ((q, x[:, :h], f64(w)), (k, x[:, h:h + 1], None)):
        want, mag = attention.norm_rope(part, wt, pos, f64(f), 1e-6, inter)
        check_norm_rope(got, want, mag, t)
    q2, k2 = gdn.qk_norm_rope(qkv, h, hkv, on(cu), w, None, f, on(np.array(kv, np.int32)),
                              interleaved=inter)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    v = qkv.view(T, 4, d)[:, 3:]
    for i in range(n):
        for pool, rows in ((kp, k), (vp, v)):
            have = pool[table[i, 0]:table[i, 0] + need[i]].transpose(1, 2).reshape(-1, hkv, d)
            old = kv[i] - lens[i]
            assert torch.equal(have[old:kv[i]], rows[cu[i]:cu[i + 1]])
            assert (have[:old] == MARK).all() and (have[kv[i]:] == MARK).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("qn,kn", [(True, False), (False, True), (False, False)])
def test_norm_rope_without_norms_and_from_wider_rows(t, qn, kn):
    """Norms are optional each; positions count from 0 without kv_lens; the packed
    rows may lie inside wider ones."""
    T, h, hkv, d, rot = 70, 4, 4, 128, 96
    wide = normal(3, T, 12 * d + 40, dtype=t).to(DEV)
    qkv = wide[:, 16:16 + 12 * d]
    w = normal(4, d, dtype=torch.float32)
    f = gdn.rope_inv_freq(rot, 1e6)
    cu = cu_of([60, 10])
    q, k = gdn.qk_norm_rope(qkv, h, hkv, on(cu), w.to(DEV) if qn else None,
                            w.to(DEV) if kn else None, f.to(DEV))
    x = f64(qkv).reshape(T, 12, d)
    for got, part, norm in ((q, x[:, :h], qn), (k, x[:, h:2 * h], kn)):
        want, mag = attention.norm_rope(part, f64(w) if norm else None, attention.positions(cu),
                                        f64(f), 1e-6)
        check_norm_rope(got, want, mag, t)


def test_norm_rope_of_zero_rows_and_values_that_are_not_finite():
    """A zero head stays zero (eps); NaN and infinities stay in their own head."""
    d = 128
    x = normal(5, 4, 3 * d)
    x[0, :d] = 0
    x[1, d + 3] = float("nan")
    x[2, 5] = float("inf")
    q, k = gdn.qk_norm_rope(x.to(DEV), 1, 1, on(cu_of([4])), torch.ones(d, device=DEV),
                            torch.ones(d, device=DEV), gdn.rope_inv_freq(d).to(DEV))
    q, k = f64(q), f64(k)
    assert np.all(q[0] == 0) and not np.isfinite(k[1]).all() and not np.isfinite(q[2]).all()
    assert np.isfinite(q[[1, 3]]).all() and np.isfinite(k[[0, 2, 3]]).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,page,inter,rot", [(128, 16, False, 128), (256, 64, True, 64),
                                              (128, 256, False, 30), (256, 32, False, 256)])
def test_append(t, d, page, inter, rot):
    """Rows land in their pages, everything else in the pool stays as it was, and
    q, k are those of the plain pass bit for bit."""
    lens, h, hkv = [1, 0, 37, 5, 1], 4, 2
    kv = [1, 3, 37 + 30, 5 + page - 2, 300]
    T, n = sum(lens), len(lens)
    c = Cache(kv, hkv, d, page, t, 11)
    cu = cu_of(lens)
    qkv = normal(12, T + 3, (h + 2 * hkv) * d, dtype=t).to(DEV)
    w = normal(13, d, dtype=torch.float32).to(DEV)
    f = gdn.rope_inv_freq(rot).to(DEV)
    kp, vp = c.k.to(DEV), c.v.to(DEV)
    say(f"append {t} d={d} page={page} rot={rot}")
    cfg = gdn.make_attn_config(T + 3, n, h, hkv, d, t, rot_dim=rot, rot_interleaved=inter,
                               page_size=page, n_pages=c.n_pages, max_pages=c.cols)
    q = torch.full((T + 3, h, d), MARK, dtype=t, device=DEV)
    k = torch.full((T + 3, hkv, d), MARK, dtype=t, device=DEV)
    args = (cfg, qkv, w, w, f, on(cu), on(np.array(kv, np.int32)))
    gdn.gdn_kv_append(*args, on(c.table), q, k, kp, vp)
    q2, k2 = torch.full_like(q, MARK), torch.full_like(k, MARK)
    gdn.gdn_qk_norm_rope(*args, q2, k2)
    assert torch.equal(q, q2) and torch.equal(k, k2) and (q[T:] == MARK).all()
    want_k, want_v = c.k.clone(), c.v.clone()
    v = qkv.view(T + 3, h + 2 * hkv, d)[:, h + hkv:].cpu()
    row = 0
    for s in range(n):
        for p in range(kv[s] - lens[s], kv[s]):
            want_k[c.table[s, p // page], :, p % page] = k[row].cpu()
            want_v[c.table[s, p // page], :, p % page] = v[row]
            row += 1
    bits = lambda x: x.cpu().view(torch.int16)  # noqa: E731  (NaN included)
    assert torch.equal(bits(kp), bits(want_k)) and torch.equal(bits(vp), bits(want_v))
    # the pages alone, neither q nor k wanted
    kp3, vp3 = c.k.to(DEV), c.v.to(DEV)
    gdn.gdn_kv_append(*args, on(c.table), None, None, kp3, vp3)
    assert torch.equal(bits(kp3), bits(kp)) and torch.equal(bits(vp3), bits(vp))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 34, False), (256, 64, True)])
def test_a_large_append_equals_its_halves(t, d, rot, inter):
    """More than 256 MiB written in one call (outputs past the caches), against the same
    sequence appended in two, which are small enough for them."""
    h, hkv, page = 2, 1, 256
    T = (280 << 20) // ((h + 3 * hkv) * d * 2) // 2 * 2
    x = torch.randn(T, (h + 2 * hkv) * d, device=DEV).to(t)
    w, f = normal(31, d, dtype=torch.float32).to(DEV), gdn.rope_inv_freq(rot).to(DEV)
    pages = -(-T // page)
    table = torch.randperm(pages, device=DEV).to(torch.int32)[None]
    kp = torch.full((pages, hkv, page, d), MARK, dtype=t, device=DEV)
    vp, k2, v2 = kp.clone(), kp.clone(), kp.clone()
    say(f"large append {t} T={T} d={d}")

    def append(rows, end, kp, vp):
        n = rows.shape[0]
        return gdn.append_paged_kv(rows, h, on(cu_of([n])), on(np.array([end], np.int32)), table, kp,
                                   vp, w, w, f, interleaved=inter, output_k=True)

    q, k = append(x, T, kp, vp)
    parts = [append(x[:T // 2], T // 2, k2, v2), append(x[T // 2:], T, k2, v2)]
    assert torch.equal(q, torch.cat([y[0] for y in parts]))
    assert torch.equal(k, torch.cat([y[1] for y in parts]))
    assert torch.equal(kp, k2) and torch.equal(vp, v2)
    torch.cuda.empty_cache()


def test_append_skips_rows_without_a_page():
    """Entries that name no page, columns past the table and negative positions."""
    t, d, page, hkv = torch.bfloat16, 128, 16, 1
    lens = [2, 2, 2, 3]
    kv = np.array([2, 2, 50, 1], np.int32)  # 50: column 3 of 2; 1: two positions below zero
    table = np.array([[-1, 0], [7, 0], [1, 2], [3, 3]], np.int32)  # 4 pages: 7 names none
    pool = torch.full((4, hkv, page, d), MARK, dtype=t, device=DEV)
    kp, vp = pool.clone(), pool.clone()
    q = gdn.append_paged_kv(normal(1, 9, 3 * d, dtype=t).to(DEV), 1, on(cu_of(lens)), on(kv),
                            on(table), kp, vp)
    touched = (kp != MARK).any(-1).nonzero().tolist()
    assert touched == [[3, 0, 0]] and (vp != MARK).any(-1).nonzero().tolist() == [[3, 0, 0]]
    assert q.isfinite().all()


# ---------------------------------------------------------------- prefill

PREFILL = [
    # new tokens, tokens in all of each sequence; h, hkv, d
    ([1], [1], 1, 1, 128),
    ([1], [200], 8, 2, 256),
    ([64], [64], 2, 2, 128),
    ([65, 63], [65, 63], 4, 1, 128),
    ([127, 0, 129, 1], [127, 5, 129, 1], 4, 2, 256),
    ([300], [300], 3, 1, 128),
    ([100, 33, 2], [228, 161, 500], 4, 4, 128),
    ([9, 40, 5], [0, 17, 5], 2, 1, 128),     # rows that see no key
    ([200, 140], [130, 40], 2, 1, 256),      # whole tiles that see no key
    ([260], [260], 16, 1, 128),
    ([70, 1], [110, 41], 5, 1, 128),          # queries that start inside a tile of keys
    ([150], [190], 2, 2, 256),
    ([40], [3000], 8, 2, 128),                # few rows and many keys: split
    ([3], [2500], 4, 1, 256),
    ([12, 7], [0, 2100], 6, 2, 128),
    ([140], [140], 17, 1, 128),               # a prime number of heads on one key head
    ([50, 33], [90, 40], 24, 1, 256),
    ([30], [40], 64, 2, 128),
    ([2], [9], 4096, 1, 128),                 # the most heads
    ([i % 4 for i in range(100)], [520 + 5 * i for i in range(100)], 1, 1, 128),  # parts, many sequences
]


def _poisoned(x, cu, rows):
    """Rows of x behind the last sequence hold NaN."""
    x = x.clone()
    x[int(cu[-1]):rows] = float("nan")
    return x


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("new,full,h,hkv,d", PREFILL)
def test_prefill(t, new, full, h, hkv, d):
    T, Tk, n = sum(new) + 5, sum(full) + 3, len(new) + 2
    cu_q, cu_k = cu_of(new, n), cu_of(full, n)
    q = _poisoned(normal(1, T, h, d, dtype=t, scale=2.0), cu_q, T)
    kv = _poisoned(normal(2, Tk, 2 * hkv, d, dtype=t), cu_k, Tk)
    k, v = kv[:, :hkv].contiguous(), kv[:, hkv:]
    say(f"prefill {t} {new} of {full} h={h} hkv={hkv} d={d}")
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, tk_max=Tk)
    o = torch.full((T, h, d), MARK, dtype=t, device=DEV)
    kv_dev = kv.to(DEV)  # v is read inside its wider rows
    gdn.gdn_attn_prefill(cfg, q.to(DEV), k.to(DEV), kv_dev[:, hkv:], on(cu_q), on(cu_k), o,
                         workspace(cfg))
    worst = 0.0
    for s in range(len(new)):
        a, b = slice(cu_q[s], cu_q[s + 1]), slice(cu_k[s], cu_k[s + 1])
        worst = max(worst, check_attention(o[a], f64(q[a]), f64(k[b]), f64(v[b]), d ** -0.5, t))
    say(f"  off / bound {worst:.3f}")
    assert (o[sum(new):] == MARK).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("T,past,h,hkv,d", [(4500, 0, 2, 1, 128), (2100, 25, 1, 1, 256),
                                            (1500, 2011, 4, 1, 128)])
def test_prefill_of_long_prompts_at_sampled_rows(t, T, past, h, hkv, d):
    """Every 97th row and the last one against the oracle; every row finite, and of
    the size of a mean of values."""
    q = normal(1, T, h, d, dtype=t, scale=2.0)
    k, v = (normal(i, T + past, hkv, d, dtype=t) for i in (2, 3))
    say(f"prefill {t} {T} of {T + past} h={h} d={d}")
    o = gdn.causal_attention(q.to(DEV), k.to(DEV), v.to(DEV), on(cu_of([T])),
                             on(cu_of([T + past])))
    assert o.isfinite().all() and float(o.abs().max()) <= float(v.abs().max()) * 1.01
    for r in [*range(0, T, 97), T - 1]:
        check_attention(o[r:r + 1], f64(q[r:r + 1]), f64(k[:past + r + 1]), f64(v[:past + r + 1]),
                        d ** -0.5, t)


@pytest.mark.parametrize("t", TYPES)
def test_prefill_of_the_same_tokens_and_a_caller_scale(t):
    T, h, hkv, d = 150, 4, 2, 128
    q, k, v = (normal(i, T, n, d, dtype=t) for i, n in ((1, h), (2, hkv), (3, hkv)))
    o = gdn.causal_attention(q.to(DEV), k.to(DEV), v.to(DEV), on(cu_of([150])), scale=0.5)
    check_attention(o, f64(q), f64(k), f64(v), 0.5, t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("big", [1.0, 60.0])
def test_prefill_of_scores_that_grow_along_the_keys(t, big):
    """The running maximum moves at every tile, by little and by much."""
    T, d = 400, 128
    q = torch.ones(T, 1, d, dtype=t)
    k = (torch.linspace(-1, 1, T)[:, None, None] * big).expand(T, 1, d).to(t).contiguous()
    v = normal(7, T, 1, d, dtype=t)
    for flip in (False, True):
        kk = k.flip(0) if flip else k
        o = gdn.causal_attention(q.to(DEV), kk.to(DEV), v.to(DEV), on(cu_of([T])))
        check_attention(o, f64(q), f64(kk), f64(v), d ** -0.5, t)


def test_prefill_of_scores_at_the_types_lowest_value():
    """Keys that a caller pushed away with the lowest value of the type weigh
    nothing beside others, and all the same where there are only such."""
    t, T, d = torch.bfloat16, 70, 128
    q = torch.zeros(T, 1, d, dtype=t)
    q[..., 0] = 1.0
    k = torch.zeros(T, 1, d, dtype=t)
    k[:40, :, 0] = torch.finfo(t).min
    v = normal(8, T, 1, d, dtype=t)
    o = gdn.causal_attention(q.to(DEV), k.to(DEV), v.to(DEV), on(cu_of([T])))
    check_attention(o, f64(q), f64(k), f64(v), d ** -0.5, t)


def test_prefill_keeps_what_is_not_finite_in_its_sequence():
    t, d, lens = torch.float16, 128, [70, 64, 30]
    T = sum(lens)
    q, k, v = (normal(i, T, 1, d, dtype=t) for i in (1, 2, 3))
    k[100], v[110] = float("nan"), float("inf")  # both in the middle sequence
    o = f64(gdn.causal_attention(q.to(DEV), k.to(DEV), v.to(DEV), on(cu_of(lens))))
    assert np.isfinite(o[:70]).all() and np.isfinite(o[134:]).all()
    assert np.isnan(o[100:134]).any(-1).all()
    for a, b in ((0, 70), (134, 164)):
        check_attention(torch.from_numpy(o[a:b]).to(t), f64(q[a:b]), f64(k[a:b]), f64(v[a:b]),
                        d ** -0.5, t)


# ---------------------------------------------------------------- paged

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
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("new,full,h,hkv,d,page,shared", PAGED)
def test_paged(t, new, full, h, hkv, d, page, shared):
    T, n = sum(new) + 2, len(new) + 1
    c = Cache(list(full) + [0], hkv, d, page, t, 21, shared=shared)
    cu = cu_of(new, n)
    q = _poisoned(normal(1, T, h, d, dtype=t, scale=2.0), cu, T)
    say(f"paged {t} n={len(new)} tokens={sum(new)} keys={sum(full)} h={h} hkv={hkv} d={d} "
        f"page={page} shared={shared}")
    # a prefix, with a capacity that is too small for a pass of its own and with a larger one
    for cols in [c.cols] + ([shared_cols(n, hkv, d, page)] if shared else []):
        cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=c.n_pages,
                                   max_pages=cols, shared_max=cols * page if shared else 0)
        o = torch.full((T, h, d), MARK, dtype=t, device=DEV)
        sh = on(np.array([shared], np.int32)) if shared else None
        args = (q.to(DEV), c.k.to(DEV), c.v.to(DEV), on(cu), on(np.array(c.lens, np.int32)),
                on(widened(c.table, cols)))
        gdn.gdn_attn_paged(cfg, *args, sh, o, workspace(cfg))
        worst = 0.0
        for s in range(len(new)):
            a = slice(cu[s], cu[s + 1])
            k, v = c.rows(s)
            worst = max(worst, check_attention(o[a], f64(q[a]), k, v, d ** -0.5, t))
        say(f"  off / bound {worst:.3f}")
        assert (o[sum(new):] == MARK).all()
    # the same bits again, with another workspace's content
    o2 = torch.full_like(o, MARK)
    gdn.gdn_attn_paged(cfg, *args, sh, o2, torch.zeros_like(workspace(cfg)))
    assert torch.equal(o, o2)


@pytest.mark.parametrize("t", TYPES)
def test_paged_of_one_long_context(t):
    """One sequence split over the whole device and joined."""
    n, h, hkv, d, page = 20000, 4, 1, 128, 16
    c = Cache([n], hkv, d, page, t, 31)
    q = normal(1, 1, h, d, dtype=t, scale=3.0)
    o = gdn.paged_attention(q.to(DEV), c.k.to(DEV), c.v.to(DEV), on(cu_of([1])),
                            on(np.array([n], np.int32)), on(c.table))
    k, v = c.rows(0)
    check_attention(o, f64(q), k, v, d ** -0.5, t)


@pytest.mark.parametrize("new,full,h,hkv,d,page,shared", [
    ([1, 1], [9000, 700], 8, 2, 128, 16, 0),                 # keys in parts, four waves per row
    ([1] * 300, [100 + 3 * i for i in range(300)], 16, 4, 128, 32, 0),  # and one wave per row
    ([1, 2, 1], [900, 950, 1200], 16, 2, 256, 16, 700),      # beside a shared prefix
    ([200, 40], [500, 40], 8, 2, 128, 16, 0),                # tiles over the pages
    ([140], [4000], 4, 2, 256, 64, 0),                       # with their keys in parts
])
def test_paged_keeps_what_is_not_finite_in_its_rows(new, full, h, hkv, d, page, shared):
    """NaN in a query row, or +inf in a cached value, comes out of the rows that read it
    and of no other sequence's."""
    t = torch.bfloat16
    c = Cache(full, hkv, d, page, t, 3, shared)
    q = normal(1, sum(new), h, d, dtype=t)
    q[0, 0] = float("nan")
    last = len(new) - 1
    at = full[last] - 1 - new[last] // 2  # the last sequence's, behind the prefix
    c.v[c.table[last, at // page], :, at % page] = float("inf")
    args = [x.to(DEV) for x in (q, c.k, c.v)]
    sh = torch.tensor([shared], dtype=torch.int32, device=DEV) if shared else None
    cu = cu_of(new)
    say(f"paged, values that are not finite {new[:4]} {full[:4]} d={d} shared={shared}")
    table = widened(c.table, shared_cols(len(new), hkv, d, page)) if shared else c.table
    o = gdn.paged_attention(*args, on(cu), on(np.array(full, np.int32)), on(table), sh)
    assert o[0, 0].isnan().all()
    b = int(cu[last]) if last else 0
    if last:
        assert o[:b].flatten(0, 1)[1:].isfinite().all()
    reads = full[last] - new[last] + np.arange(new[last]) >= at
    assert not o[b:][torch.from_numpy(reads).to(DEV)].isfinite().any()


@pytest.mark.parametrize("d,hkv", [(128, 8), (256, 4)])
def test_paged_of_more_keys_than_the_caches_hold(d, hkv):
    """66000 keys of 4096 bytes, read past the caches: a streamed row and tiles in parts."""
    t, h, T, lens = torch.bfloat16, 4 * hkv, 20, [66000, 300]
    c = Cache(lens, hkv, d, 256, t, 17)
    kp, vp, table, kv = c.k.to(DEV), c.v.to(DEV), on(c.table), on(np.array(lens, np.int32))
    q = normal(5, T + 1, h, d, dtype=t)
    for new in ([1, 1], [T, 1]):
        say(f"more keys than the caches hold d={d} new={new}")
        cu = cu_of(new)
        o = gdn.paged_attention(q[:sum(new)].to(DEV), kp, vp, on(cu), kv, table)
        for s in range(2):
            a = slice(cu[s], cu[s + 1])
            check_attention(o[a], f64(q[a]), *c.rows(s), d ** -0.5, t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("T,past,d", [(2100, 333, 128), (700, 900, 256)])
def test_paged_of_a_long_prompt_at_sampled_rows(t, T, past, d):
    h, hkv, page = 2, 1, 64
    c = Cache([T + past], hkv, d, page, t, 33)
    q = normal(1, T, h, d, dtype=t, scale=2.0)
    o = gdn.paged_attention(q.to(DEV), c.k.to(DEV), c.v.to(DEV), on(cu_of([T])),
                            on(np.array([T + past], np.int32)), on(c.table))
    k, v = c.rows(0)
    assert o.isfinite().all()
    for r in [*range(0, T, 131), T - 1]:
        check_attention(o[r:r + 1], f64(q[r:r + 1]), k[:past + r + 1], v[:past + r + 1], d ** -0.5, t)


def test_both_capacity_limits_with_sequences_at_the_end():
    """t_max = 2^24 rows and n_max = 16384 sequences, the checked ones the last two
    (byte offsets far past 2^32): front, prefill and paged attention."""
    t, d, h, hkv = torch.bfloat16, 128, 1, 1
    T, n, page = gdn.GDN_T_MAX_LIMIT, gdn.GDN_N_MAX_LIMIT, 256
    tail = [70, 3]
    cu = np.zeros(n + 1, np.int64)
    cu[:n - 1] = np.linspace(0, T - sum(tail), n - 1).astype(np.int64)
    cu[n - 1:] = T - tail[1], T
    say(f"capacity limits: {T} rows, {n} sequences")
    x = torch.zeros(T, 3 * d, dtype=t, device=DEV)
    x[T - sum(tail):] = normal(1, sum(tail), 3 * d, dtype=t).to(DEV)
    f, w = gdn.rope_inv_freq(d).to(DEV), torch.ones(d, device=DEV)
    cud = on(cu.astype(np.int32))
    q, k = gdn.qk_norm_rope(x, h, hkv, cud, w, w, f)
    xs = f64(x[-sum(tail):]).reshape(-1, 3, d)
    pos = np.concatenate([np.arange(70.0), np.arange(3.0)])
    for got, part in ((q, xs[:, :1]), (k, xs[:, 1:2])):
        want, mag = attention.norm_rope(part, np.ones(d), pos, f64(f), 1e-6)
        check_norm_rope(got[-sum(tail):], want, mag, t)
        assert not got[:T - sum(tail)].any()
    v = x.view(T, 3, d)[:, 2:]
    o = gdn.causal_attention(q, k, v, cud)
    for a, b in ((T - 73, T - 3), (T - 3, T)):
        check_attention(o[a:b], f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), d ** -0.5, t)
    assert not o[:T - sum(tail)].any()
    del x, o, v
    # the paged side: one row per sequence, all tables in a small pool
    c = Cache([300, 41], hkv, d, page, t, 5)
    table = np.zeros((n, c.cols), np.int32)
    table[n - 2:] = c.table
    kv = np.ones(n, np.int32)
    kv[n - 2:] = c.lens
    qq = torch.zeros(n, h, d, dtype=t, device=DEV)
    qq[n - 2:] = normal(6, 2, h, d, dtype=t).to(DEV)
    vp = c.v.clone()
    vp[0, :, 0] = torch.where(vp[0, :, 0].isnan(), torch.zeros_like(vp[0, :, 0]), vp[0, :, 0])
    kp = c.k.clone()
    kp[0, :, 0] = torch.where(kp[0, :, 0].isnan(), torch.zeros_like(kp[0, :, 0]), kp[0, :, 0])
    o = gdn.paged_attention(qq, kp.to(DEV), vp.to(DEV), on(np.arange(n + 1, dtype=np.int32)),
                            on(kv), on(table))
    assert torch.equal(o[:n - 2, 0], vp[0, 0, 0].to(DEV).expand(n - 2, d))
    c.k, c.v = kp, vp
    for i in range(2):
        rk, rv = c.rows(i)
        check_attention(o[n - 2 + i:n - 1 + i], f64(qq[n - 2 + i:n - 1 + i]), rk, rv, d ** -0.5, t)
    del q, k
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [128, 256])
def test_prefill_of_rows_as_far_apart_as_they_may_be(d):
    """k and v rows 2^24 elements apart: a tile's last offset is just below 2^31 bytes."""
    t, T, far = torch.bfloat16, 100, 1 << 24
    q, k, v = (normal(i, T, 1, d, dtype=t) for i in (1, 2, 3))
    say(f"rows 2^24 apart d={d}")
    buf = torch.zeros((T - 1) * far + 2 * d, dtype=t, device=DEV)
    kd, vd = (buf[at:].as_strided((T, 1, d), (far, d, 1)) for at in (0, d))
    kd.copy_(k.to(DEV)), vd.copy_(v.to(DEV))
    o = gdn.causal_attention(q.to(DEV), kd, vd, on(cu_of([T])))
    check_attention(o, f64(q), f64(k), f64(v), d ** -0.5, t)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [128, 256])
def test_batches_without_tokens_write_nothing(d):
    t, h, hkv, page, n, T = torch.float16, 4, 2, 16, 3, 9
    kp = torch.full((5, hkv, page, d), MARK, dtype=t, device=DEV)
    vp, cu = kp.clone(), on(np.zeros(n + 1, np.int32))
    kv, table = on(np.full(n, 20, np.int32)), on(np.zeros((n, 2), np.int32))
    x = normal(1, T, (h + 2 * hkv) * d, dtype=t).to(DEV)
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=5, max_pages=2)
    q, o = (torch.full((T, h, d), MARK, dtype=t, device=DEV) for _ in range(2))
    k = torch.full((T, hkv, d), MARK, dtype=t, device=DEV)
    gdn.gdn_qk_norm_rope(cfg, x, None, None, None, cu, None, q, k)
    gdn.gdn_kv_append(cfg, x, None, None, None, cu, kv, table, q, k, kp, vp)
    gdn.gdn_attn_prefill(cfg, q, k, k, cu, None, o, workspace(cfg))
    gdn.gdn_attn_paged(cfg, q, kp, vp, cu, kv, table, None, o, workspace(cfg))
    for y in (q, k, o, kp, vp):
        assert (y == MARK).all()


def test_paged_indexes_that_name_nothing_stay_inside():
    """Lengths past the table, entries past the pool and a decreasing cu_seqlens
    give some values, and write only rows of o."""
    t, h, hkv, d, page = torch.bfloat16, 4, 1, 128, 16
    n, T, pages = 5, 12, 3
    kp, vp = normal(1, pages, hkv, page, d).to(DEV), normal(2, pages, hkv, page, d).to(DEV)
    table = np.array([[0, 1], [-5, 9], [2_000_000_000, 1], [1, -2_000_000_000], [2, 2]], np.int32)
    buf = torch.full((T + 8, h, d), MARK, dtype=t, device=DEV)
    q, sh = normal(3, T, h, d).to(DEV), on(np.array([1 << 30], np.int32))
    for cols in (2, shared_cols(n, hkv, d, page)):
        cfg = gdn.make_attn_config(T, n, h, hkv, d, t, page_size=page, n_pages=pages, max_pages=cols,
                                   shared_max=64 if cols == 2 else 1 << 30)
        wide = on(widened(table, cols))
        for cu in ([0, 2, 3, 9, 10, 12], [0, 9, 4, 4, 20, 11], [5, 3, -7, 12, 1, 40]):
            for kv in ([32, 31, 20, 2_000_000_000, 0], [-4, 1000, 32, 32, 32]):
                gdn.gdn_attn_paged(cfg, q, kp, vp, on(np.array(cu, np.int32)),
                                   on(np.array(kv, np.int32)), wide, sh, buf[4:4 + T],
                                   workspace(cfg))
                assert (buf[:4] == MARK).all() and (buf[4 + T:] == MARK).all()


def test_prefill_and_front_with_malformed_cu_seqlens_stay_inside():
    t, h, hkv, d, T, n = torch.bfloat16, 2, 1, 128, 40, 3
    cfg = gdn.make_attn_config(T, n, h, hkv, d, t, rot_dim=64)
    x = normal(1, T, 4 * d).to(DEV)
    f, w = gdn.rope_inv_freq(64).to(DEV), torch.ones(d, device=DEV)
    bufs = [torch.full((T + 8, m, d), MARK, dtype=t, device=DEV) for m in (h, hkv, h)]
    q, k, o = (b[4:4 + T] for b in bufs)
    for cu in ([0, 30, 10, 40], [0, -5, 90, 20], [7, 7, 60, 41]):
        c = on(np.array(cu, np.int32))
        gdn.gdn_qk_norm_rope(cfg, x, w, w, f, c, None, q, k)
        gdn.gdn_attn_prefill(cfg, x[:, :h * d], x[:, h * d:(h + 1) * d], x[:, (h + 1) * d:], c, None,
                             o, workspace(cfg))
        for b in bufs:
            assert (b[:4] == MARK).all() and (b[4 + T:] == MARK).all()


# ---------------------------------------------------------------- as they are used together

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,page,rot,inter", [(128, 16, 128, False), (256, 64, 64, True)])
def test_prompt_then_steps(t, d, page, rot, inter):
    """Two prompts that begin alike: norm, rotation and append, attention over the
    prompt, then decode and verify steps over the cache with the shared pages
    read once; every output against the oracle on the q, k, v that went in."""
    h, hkv, common = 8, 2, 70
    lens = [90, 75]
    steps = [[1, 1], [3, 0], [2, 4]]
    total = [lens[i] + sum(s[i] for s in steps) for i in range(2)]
    sp = common // page
    need = [-(-x // page) for x in total]
    pages = sp + sum(x - sp for x in need)
    table = np.full((2, max(need)), -1, np.int32)
    table[0, :need[0]] = range(need[0])
    table[1, :need[1]] = list(range(sp)) + list(range(need[0], pages))
    kp = torch.full((pages, hkv, page, d), float("nan"), dtype=t, device=DEV)
    vp = kp.clone()
    w = [normal(i, d, dtype=torch.float32, scale=0.3).add(1.0).to(DEV) for i in (1, 2)]
    f = gdn.rope_inv_freq(rot, 1e6, factor=4.0, original_len=64).to(DEV)
    width = (h + 2 * hkv) * d
    same = normal(40, common, width, dtype=t)
    prompt = torch.cat([same, normal(41, lens[0] - common, width, dtype=t),
                        same, normal(42, lens[1] - common, width, dtype=t)]).to(DEV)
    history = [[[], []], [[], []]]  # k, v rows of each sequence as the cache should have them

    def front(x, cu, kv):
        q, k = gdn.append_paged_kv(x, h, on(cu), on(np.array(kv, np.int32)), on(table), kp, vp,
                                   w[0], w[1], f, interleaved=inter, output_k=True)
        xs = f64(x).reshape(-1, h + 2 * hkv, d)
        pos = attention.positions(cu, kv)
        for got, part, wt in ((q, xs[:, :h], w[0]), (k, xs[:, h:h + hkv], w[1])):
            want, mag = attention.norm_rope(part, f64(wt), pos, f64(f), 1e-6, inter)
            check_norm_rope(got, want, mag, t)
        for s in range(2):
            a = slice(cu[s], cu[s + 1])
            history[s][0].append(f64(k[a]))
            history[s][1].append(xs[a, h + hkv:])
        return q, k

    cu, kv = cu_of(lens), list(lens)
    q, k = front(prompt, cu, kv)
    v = prompt.view(-1, h + 2 * hkv, d)[:, h + hkv:]
    o = gdn.causal_attention(q, k, v, on(cu))
    po = gdn.paged_attention(q, kp, vp, on(cu), on(np.array(kv, np.int32)), on(table))
    for s in range(2):
        a = slice(cu[s], cu[s + 1])
        for out in (o, po):
            check_attention(out[a], f64(q[a]), history[s][0][0], history[s][1][0], d ** -0.5, t)
    shared = on(np.array([common], np.int32))
    for i, new in enumerate(steps):
        cu = cu_of(new)
        kv = [kv[s] + new[s] for s in range(2)]
        q, _ = front(normal(50 + i, sum(new), width, dtype=t).to(DEV), cu, kv)
        wide = widened(table, shared_cols(2, hkv, d, page))
        o = gdn.paged_attention(q, kp, vp, on(cu), on(np.array(kv, np.int32)), on(wide), shared)
        for s in range(2):
            a = slice(cu[s], cu[s + 1])
            check_attention(o[a], f64(q[a]), np.concatenate(history[s][0]),
                            np.concatenate(history[s][1]), d ** -0.5, t)


def test_a_captured_decode_step_replays_with_other_lengths():
    """append + paged attention in one graph: lengths, tables and the shared length
    are read on the device, so one capture serves every step."""
    t, h, hkv, d, page, n = torch.bfloat16, 8, 2, 128, 16, 6
    rng = np.random.Generator(np.random.PCG64(3))
    cols, most = 40, shared_cols(n, hkv, d, page)
    pages = n * cols
    table = on(widened(rng.permutation(pages).reshape(n, cols).astype(np.int32), most))
    kp, vp = normal(1, pages, hkv, page, d).to(DEV), normal(2, pages, hkv, page, d).to(DEV)
    cfg = gdn.make_attn_config(2 * n, n, h, hkv, d, t, rot_dim=128, page_size=page, n_pages=pages,
                               max_pages=most, shared_max=most * page)
    x = torch.zeros(2 * n, (h + 2 * hkv) * d, dtype=t, device=DEV)
    cu, kv = on(cu_of([1] * n)), on(np.full(n, 5, np.int32))
    sh = on(np.array([0], np.int32))
    f, w = gdn.rope_inv_freq(128).to(DEV), torch.ones(d, device=DEV)
    q, o = (torch.zeros(2 * n, h, d, dtype=t, device=DEV) for _ in range(2))

    def step(q, o, kp, vp, ws):
        gdn.gdn_kv_append(cfg, x, w, w, f, cu, kv, table, q, None, kp, vp)
        gdn.gdn_attn_paged(cfg, q, kp, vp, cu, kv, table, sh, o, ws)

    ws = workspace(cfg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q, o, kp, vp, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q, o, kp, vp, ws)
    for i in range(6):
        new = [1] * n if i % 2 == 0 else [0, 2, 3, 1, 4, 2]
        cu.copy_(on(cu_of(new)))
        kv.copy_(on(rng.integers(200, cols * page, n).astype(np.int32)))
        table[:, :12] = table[0, :12] if i in (2, 3) else table[:, :12]
        sh.fill_(170 if i in (2, 3) else 0)
        x.copy_(normal(60 + i, *x.shape))
        q2, o2, k2, v2 = torch.zeros_like(q), torch.zeros_like(o), kp.clone(), vp.clone()
        o.zero_(), q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        step(q2, o2, k2, v2, workspace(cfg))
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(q, q2), i
        assert torch.equal(kp, k2) and torch.equal(vp, v2), i


@pytest.mark.parametrize("d", [128, 256])
def test_two_graphs_that_share_a_workspace(d):
    """Split prefill, a prompt over pages and a decode step, captured apart with one
    workspace and replayed in turn: nothing in it outlives a call."""
    t, h, hkv, page = torch.bfloat16, 8, 2, 32
    c = Cache([1500, 260], hkv, d, page, t, 90)
    kp, vp, table = c.k.to(DEV), c.v.to(DEV), on(c.table)
    kv, tail = on(np.array(c.lens, np.int32)), on(cu_of([1, 1]))
    q = normal(91, 300, h, d, dtype=t).to(DEV)
    k, v = (normal(92 + i, 1900, hkv, d, dtype=t).to(DEV) for i in range(2))
    cu, cuk = on(cu_of([100, 200])), on(cu_of([900, 1000]))
    cfgs = [gdn.make_attn_config(300, 2, h, hkv, d, t, tk_max=1900),
            gdn.make_attn_config(300, 2, h, hkv, d, t, page_size=page, n_pages=c.n_pages,
                                 max_pages=c.cols),
            gdn.make_attn_config(2, 2, h, hkv, d, t, page_size=page, n_pages=c.n_pages,
                                 max_pages=c.cols)]
    calls = [lambda o, ws: gdn.gdn_attn_prefill(cfgs[0], q, k, v, cu, cuk, o, ws),
             lambda o, ws: gdn.gdn_attn_paged(cfgs[1], q, kp, vp, cu, kv, table, None, o, ws),
             lambda o, ws: gdn.gdn_attn_paged(cfgs[2], q[:2], kp, vp, tail, kv, table, None, o[:2], ws)]
    want = []
    for cfg, call in zip(cfgs, calls):
        want.append(torch.zeros_like(q))
        call(want[-1], workspace(cfg))
    ws = torch.empty(max(gdn.gdn_attn_workspace_size(x) for x in cfgs), dtype=torch.uint8, device=DEV)
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
        c = Cache([3000 + 500 * i, 40], hkv, d, page, t, 70 + i)
        q = normal(80 + i, 2, h, d, dtype=t).to(DEV)
        runs.append((q, c.k.to(DEV), c.v.to(DEV), on(cu_of([1, 1])),
                     on(np.array(c.lens, np.int32)), on(c.table)))
    alone = [gdn.paged_attention(*r) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        outs = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                outs.append(gdn.paged_attention(*r))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))


def test_offsets_past_32_bits_in_a_large_pool():
    """Pages whose byte offsets pass 2^32, written by append and read by attention."""
    t, h, hkv, d, page = torch.bfloat16, 4, 2, 256, 256
    pages = 9000  # 9000 * 2 * 256 * 256 * 2 bytes: 2.4e9 values
    kp = torch.zeros(pages, hkv, page, d, dtype=t, device=DEV)
    vp = torch.zeros_like(kp)
    n = 300
    table = np.array([[pages - 1, 8500]], np.int32)
    x = normal(5, n, (h + 2 * hkv) * d, dtype=t).to(DEV)
    kv, cu = on(np.array([n], np.int32)), on(cu_of([n]))
    q, k = gdn.append_paged_kv(x, h, cu, kv, on(table), kp, vp, output_k=True)
    assert torch.equal(kp[pages - 1].transpose(0, 1), k[:256])
    assert torch.equal(kp[8500, :, :44].transpose(0, 1), k[256:])
    assert not kp[8499].any() and not vp[:8500].any()
    o = gdn.paged_attention(q[-1:].contiguous(), kp, vp, on(cu_of([1])), kv, on(table))
    v = x.view(n, h + 2 * hkv, d)[:, h + hkv:]
    check_attention(o, f64(q[-1:]), f64(k), f64(v), d ** -0.5, t)
