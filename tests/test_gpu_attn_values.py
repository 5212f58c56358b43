"""Softmax attention at the ends of its types' ranges, against the fp64 oracle: weights
far below the largest, scores past the whole numbers of fp32. Every way that keys and
values are read takes each case. Bounds: attn_helpers.py, except where one is stated."""

import numpy as np
import pytest
import torch

import chunked_gated_delta_rule_amd as gdn
from attn_helpers import (DEV, check_norm_rope, cu_of, f64, half_step, normal, on, shared_cols,
                          widened)
from oracle import attention

pytestmark = pytest.mark.gpu

# new tokens, keys, query and key heads; pages (0: packed rows); sequences behind a shared
# prefix (0: one sequence)
WAYS = {
    "rows": (150, 150, 4, 2, 0, 0),           # whole tiles
    "row parts": (20, 700, 2, 1, 0, 0),       # tiles with their keys in parts, joined
    "stream": (1, 30, 4, 1, 16, 0),           # one wave's keys
    "stream parts": (2, 900, 4, 2, 16, 0),    # work-groups joined
    "pages": (80, 300, 4, 1, 32, 0),          # tiles over the pages
    "page parts": (80, 1500, 4, 1, 64, 0),
    "prefix": (2, 400, 4, 1, 16, 3),          # a prefix of 64 read once, joined with the streams
    "wide stream": (6, 500, 4, 1, 16, 0),     # items of two row tiles
    "wide prefix": (10, 400, 4, 1, 16, 3),    # and of four (heads of 128)
}


def through(way, q, k, v, scale):
    """o of one sequence's rows (of the last sequence behind a prefix)."""
    _, _, _, _, page, n = WAYS[way]
    T, Tk, (hkv, d) = len(q), len(k), k.shape[1:]
    if not page:
        return gdn.causal_attention(q.to(DEV), k.to(DEV), v.to(DEV), on(cu_of([T])),
                                    on(cu_of([Tk])), scale=scale)
    pages = -(-Tk // page)
    pool = [torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pages * page - Tk))
            .view(pages, page, hkv, d).transpose(1, 2).contiguous().to(DEV) for x in (k, v)]
    table = np.arange(pages, dtype=np.int32)[None]
    if not n:
        return gdn.paged_attention(q.to(DEV), *pool, on(cu_of([T])), on(np.array([Tk], np.int32)),
                                   on(table), scale=scale)
    table = widened(table.repeat(n, 0), shared_cols(n, hkv, d, page))
    o = gdn.paged_attention(q.repeat(n, 1, 1).to(DEV), *pool, on(cu_of([T] * n)),
                            on(np.full(n, Tk, np.int32)), on(table),
                            on(np.array([64], np.int32)), scale=scale)
    assert all(torch.equal(o[:T], o[T * i:T * (i + 1)]) for i in range(n))
    return o[-T:]


def zeros(way, d, t):
    T, Tk, h, hkv, _, _ = WAYS[way]
    return torch.zeros(T, h, d, dtype=t), torch.zeros(Tk, hkv, d, dtype=t)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("nats", [12.0, 16.0, 17.5, 20.0])
def test_a_tail_of_weights_far_below_the_largest(way, d, nats):
    """One key of great weight and a value of zero before many of little weight: the
    output is the tail's. fp16 weights are formed 2^7 times larger than the row's largest
    would have them, so a weight is off by half a step or, below the normal numbers, by
    2^-25 2^-7 of the largest. The scores are exact products of one dim (e: their one
    rounding with the scale, 2^-24 nats twice)."""
    t = torch.float16
    q, k = zeros(way, d, t)
    q[..., 0] = 1.0
    k[0, :, 0] = nats
    v = (1000.0 * (1.0 + 0.25 * normal(3, *k.shape, dtype=torch.float32))).to(t)
    v[0] = 0
    print(f"tail {way} d={d} nats={nats}", flush=True)
    got = f64(through(way, q, k, v, 1.0))
    o, mag, total = attention.attend(f64(q), f64(k), f64(v), 1.0)
    u, e = half_step(t), nats * 2.0 ** -23
    bound = 1.01 * (u * np.abs(o) + (u + 2 * e + 2.0 ** -18) * mag) + 2.0 ** -25 + \
        len(k) * 2.0 ** -32 * np.abs(f64(v)).max() / total[..., None]
    off = np.abs(got - o)
    print(f"  off / bound {np.max(off / bound):.3f}", flush=True)
    assert np.all(off <= bound), np.max(off / bound)


# values of q and of k in the first dims (so many of them), and the scale
FAR = [("lowest", torch.bfloat16, 1.0, torch.finfo(torch.bfloat16).min, 1, None),
       ("highest", torch.bfloat16, 1.0, torch.finfo(torch.bfloat16).max, 1, None),
       ("large", torch.bfloat16, 48640.0, 48640.0, 1, None),
       ("large and low", torch.bfloat16, 48640.0, -48640.0, 128, None),
       ("fp16 lowest", torch.float16, 65504.0, -65504.0, 128, None),
       ("fp16 highest", torch.float16, 65504.0, 65504.0, 128, None),
       ("fp16, one dim", torch.float16, 65504.0, 65504.0, 1, 0.75),
       ("a large scale", torch.float16, 3.0, 5.0, 1, 1e9)]


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("name,t,a,b,dims,scale", FAR)
def test_equal_scores_of_any_size_weigh_the_same(way, d, name, t, a, b, dims, scale):
    """The first 30 keys of a sequence have one score, far past where fp32 holds a score's
    fraction, the others 0 (so the former are masked, or mask). Keys of the same bits
    have scores of the same bits: they weigh exactly the same, whatever the size, and no
    term of the bound goes by it."""
    q, k = zeros(way, d, t)
    q[..., :dims] = a
    k[:30, :, :dims] = b
    v = normal(4, *k.shape, dtype=t)
    print(f"equal scores {name} {way} d={d}", flush=True)
    got = f64(through(way, q, k, v, scale))
    o, mag, total = attention.attend(f64(q), f64(k), f64(v), d ** -0.5 if scale is None else scale)
    u = half_step(t)
    bound = 1.01 * (u * np.abs(o) + (u + 2.0 ** -18) * mag) + 2.0 ** -25
    off = np.abs(got - o)
    print(f"  off / bound {np.max(off / bound):.3f}", flush=True)
    assert np.all(off <= bound), np.max(off / bound)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("t,a", [(torch.bfloat16, torch.finfo(torch.bfloat16).min),
                                 (torch.float16, 65504.0)])
def test_rows_of_far_and_of_ordinary_scores_in_one_tile(way, d, t, a):
    """Every other head's queries have far scores with the first 30 keys; the heads
    between are ordinary, and keep the usual bound. (fp16: the scale makes them far.)"""
    q, k = zeros(way, d, t)
    scale = 1.0 if t == torch.bfloat16 else 0.75
    q[:, 1::2] = normal(5, *q[:, 1::2].shape, dtype=t)
    k[:] = normal(6, *k.shape, dtype=t)
    q[..., 0] = 0
    q[:, ::2, 0] = 1.0 if t == torch.bfloat16 else a
    k[..., 0] = 0
    k[:30, :, 0] = a
    v = normal(4, *k.shape, dtype=t)
    print(f"far and ordinary {way} d={d} {t}", flush=True)
    got = through(way, q, k, v, scale / d ** 0.5)
    g, u = f64(got), half_step(t)
    o, mag, total = attention.attend(f64(q), f64(k), f64(v), scale / d ** 0.5)
    e = np.zeros(g.shape)  # the far heads' scores are exact, the others' sums are not
    e[:, 1::2] = d * 2.0 ** -24 * scale / d ** 0.5 * float(
        (q[:, 1::2].double().abs().amax((0, 1)) * k.double().abs().amax((0, 1)))[1:].sum())
    bound = 1.01 * (u * np.abs(o) + (u + 2 * e + 2.0 ** -18) * mag) + 2.0 ** -25 + \
        len(k) * 2.0 ** -32 * np.abs(f64(v)).max() / total[..., None]
    assert np.all(np.abs(g - o) <= bound)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("lens", [[5], [3, 0, 40]])
def test_prompts_without_any_key_row_give_zeros(lens, d):
    """Rows that see no key give zeros, also where the batch has no key at all; the same
    call from a captured graph."""
    t, T = torch.bfloat16, sum(lens)
    q = normal(1, T, 4, d, dtype=t).to(DEV)
    k = torch.zeros(0, 2, d, dtype=t, device=DEV)
    cu, cuk = on(cu_of(lens)), on(cu_of([0] * len(lens)))
    o = gdn.causal_attention(q, k, k.clone(), cu, cuk)
    assert o.shape == q.shape and not o.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.causal_attention(q, k, k, cu, cuk)
    for _ in range(3):
        o.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert not o.any()


# sizes of a head's values: their squares, or the sum of them, leave fp32, or are below its
# smallest normal number
SIZES = [2.0 ** 60, 2.0 ** 62, 1.9e19, 2.0 ** 90, 2.0 ** 120, 2.0 ** -52, 2.0 ** -64, 1e-25, 2.0 ** -100]


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-6])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 34, False), (256, 64, True)])
def test_norm_of_values_whose_squares_leave_fp32(d, rot, inter, eps):
    """The norm divides by the root mean square, which is of the values' own size."""
    t, h, hkv = torch.bfloat16, 4, 2
    T = len(SIZES)
    x = normal(7, T, h + 2 * hkv, d, dtype=torch.float32)
    x[:, 1:] *= torch.tensor(SIZES)[:, None, None]  # the first head as it is
    qkv = x.to(t).flatten(1)
    assert qkv.isfinite().all()
    w, f = 1.0 + 0.3 * normal(8, d, dtype=torch.float32), gdn.rope_inv_freq(rot)
    print(f"norm of large and small values d={d} rot={rot} eps={eps}", flush=True)
    q, k = gdn.qk_norm_rope(qkv.to(DEV), h, hkv, on(cu_of([T])), w.to(DEV), w.to(DEV), f.to(DEV),
                            eps=eps, interleaved=inter)
    y = f64(qkv).reshape(T, h + 2 * hkv, d)
    for got, part in ((q, y[:, :h]), (k, y[:, h:h + hkv])):
        want, mag = attention.norm_rope(part, f64(w), np.arange(T), f64(f), np.float64(np.float32(eps)),
                                        inter)
        check_norm_rope(got, want, mag, t)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_mean_of_the_largest_fp16_values_is_finite(way, d, sign):
    """Every value is the type's largest, and so is their mean. The weights of all keys but
    the first are just above the middle between two fp16 numbers: rounded, they are up
    to half a step larger than what the sum holds."""
    t = torch.float16
    q, k = zeros(way, d, t)
    q[..., 0] = 1.0
    k[1:, :, 0] = -0.67236328125  # weight 0.510501, in fp16 0.510742
    v = torch.full_like(k, sign * torch.finfo(t).max)
    print(f"largest values {way} d={d}", flush=True)
    got = f64(through(way, q, k, v, 1.0))
    bound = 1.01 * (2 * half_step(t) + 2.0 ** -18) * torch.finfo(t).max
    assert np.all(np.abs(got - f64(v)[0, 0, 0]) <= bound)
    v[0] = float("inf")
    assert not through(way, q, k, v, 1.0).isfinite().any()
