"""Softmax-attention layers served from a cache of 8-bit keys and values, and positions of
several axes: their cases, their inputs, and each operator in a plain form and in 64 bits.

  axes     the RMS norm of every query and key head and the rotation by a position of
           several axes (time, height, width of an image or video, each pair of
           channels turned by one of them), with or without the write into the pages
           of a 16-bit cache
  append8  the same pass with k and v written into the pages of an 8-bit cache: e4m3
           numbers, with one power of two for every 16 tokens of a key head. It grows
           as a block fills; the rows that were there are rounded to the new one
  attend8  attention of the new tokens of every sequence to such pages (decode,
           verify, chunks of a prompt), a prefix that the batch shares read once

q and the outputs are bfloat16 or float16, head sizes 128 and 256. `own` chooses between
the library's calls and the plain form. Pages and scales are returned as the float8
numbers that they hold (e4m3 and e8m0).
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6
BLOCK = 16  # tokens of a key head that share a scale
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# the largest number of four significant bits that each type holds: what the cache ends at
TOP = {"bf16": 1.875 * 2.0 ** 127, "fp16": 61440.0}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # five prompts of text and images: time, height and width, a quarter, three eighths and
        # three eighths of the pairs
        dict(name="axes_prompt", op="axes", n=5, tokens=8192, h=32, hkv=8, d=128, rot=128, axes=3,
             mixed=False, inter=False, past=0, page=0, type="bf16", mix=1),
        # 64 sequences verify 8 draft tokens after images, the axes taking turns along the pairs
        dict(name="axes_verify", op="axes", n=64, tokens=512, h=16, hkv=2, d=256, rot=64, axes=3,
             mixed=True, inter=False, past=20000, page=0, type="fp16", mix=2),
        # a video's tokens written into the pages of a 16-bit cache
        dict(name="axes_append", op="axes", n=2, tokens=24000, h=16, hkv=4, d=128, rot=128, axes=3,
             mixed=True, inter=True, past=100, page=32, type="bf16", mix=3),
        # one decode step of 256 sequences: one row each into blocks that are partly filled
        dict(name="append8_decode", op="append8", n=256, tokens=256, h=32, hkv=8, d=128, rot=128, axes=0,
             mixed=False, inter=False, past=2000, page=16, type="bf16", mix=4),
        # four long prompts written into pages of 64
        dict(name="append8_prompt", op="append8", n=4, tokens=32768, h=16, hkv=2, d=256, rot=64, axes=0,
             mixed=False, inter=False, past=300, page=64, type="bf16", mix=5),
        # 40 uneven chunks of text and images, positions of three axes
        dict(name="append8_axes", op="append8", n=40, tokens=2500, h=32, hkv=4, d=128, rot=128, axes=3,
             mixed=True, inter=False, past=4000, page=32, type="fp16", mix=6),
        # one user's next token
        dict(name="attend8_one", op="attend8", n=1, tokens=1, past=1000, shared=0, h=16, hkv=2, d=256,
             page=16, type="bf16", mix=7),
        # a serving batch: 256 sequences of very different lengths, one token each
        dict(name="attend8_ragged", op="attend8", n=256, tokens=256, past=4096, shared=0, h=32, hkv=8,
             d=128, page=16, type="bf16", mix=8),
        # four long contexts, eight draft tokens each
        dict(name="attend8_verify", op="attend8", n=4, tokens=32, past=60000, shared=0, h=32, hkv=4,
             d=128, page=32, type="fp16", mix=9),
        # 128 requests after one long system prompt
        dict(name="attend8_shared", op="attend8", n=128, tokens=128, past=400, shared=8192, h=16, hkv=2,
             d=256, page=64, type="fp16", mix=10),
        # one more piece of a long prompt
        dict(name="attend8_chunk", op="attend8", n=1, tokens=2048, past=9000, shared=0, h=32, hkv=8, d=128,
             page=64, type="bf16", mix=11),
        # sixteen short questions about documents that the cache holds
        dict(name="attend8_questions", op="attend8", n=16, tokens=16 * 77, past=3000, shared=0, h=16, hkv=2,
             d=256, page=128, type="bf16", mix=12),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    d = rng.choice([128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    h = hkv * rng.choice([1, 2, 4, 8] if hkv < 8 else [1, 2, 4])
    op = rng.choice(["axes", "append8", "append8", "attend8", "attend8"])
    c = dict(op=op, h=h, hkv=hkv, d=d, type=rng.choice(["bf16", "fp16"]), mix=rng.randrange(1, 1 << 20),
             page=rng.choice([16, 32, 64, 128, 256]))
    if op != "attend8":
        c["n"] = _log_int(rng, 1, 256)
        c["tokens"] = c["n"] + _log_int(rng, 1, 16000)
        c["rot"] = 2 * rng.randrange(1, d // 2 + 1)
        c["axes"] = rng.choice([1, 2, 3, 4] if op == "axes" else [0, 0, 2, 3])
        c["mixed"], c["inter"] = rng.random() < 0.5, rng.random() < 0.5
        c["past"] = _log_int(rng, 1, 2000)
        if op == "axes" and rng.random() < 0.5:
            c["page"] = 0
    else:
        new = rng.choice([1, 1, 1, 2, 5, 8, _log_int(rng, 9, 600)])
        c["n"] = _log_int(rng, 1, 128 if new <= 8 else 16)
        c["tokens"] = c["n"] * new
        c["past"] = _log_int(rng, 1, min(200000, 8000000 // new) // c["n"] + 16)
        c["shared"] = rng.choice([0, 0, _log_int(rng, 16, 8192)]) if new <= 8 else 0
    return c


def _lengths(case):
    """(new tokens, tokens in all) of each sequence: uneven, from the case alone."""
    r = random.Random(case["mix"])
    n, total = case["n"], case["tokens"]
    if case["op"] == "attend8" or total == n:  # as many tokens for every sequence
        new = [total // n] * n
    else:
        w = [r.random() + 0.01 for _ in range(n)]
        new = [1 + int((total - n) * x / sum(w)) for x in w]
        new[-1] += total - sum(new)
    past = case["past"]
    old = [case.get("shared", 0) + (r.randrange(past // 4, past + 1) if past else 0) for _ in range(n)]
    return new, [a + b for a, b in zip(new, old)]


def _places(case):
    """Positions [axes][tokens] of text with images in it: text counts on along every axis;
    an image's or a video's tokens lie at a frame, a row and a column of the place that it
    starts from, and the text goes on behind the largest of them."""
    r = random.Random(case["mix"] + 1)
    new, full = _lengths(case)
    out = []
    for a, b in zip(new, full):
        at, rows = b - a, []
        while len(rows) < a:
            if a == 1 or r.random() < 0.5:
                k = r.randrange(1, 200)
                rows += [(at + i,) * 4 for i in range(k)]
                at += k
            else:
                f, y, x = r.choice([1, 1, 4]), r.randrange(8, 40), r.randrange(8, 40)
                rows += [(at + i, at + j, at + k, at) for i in range(f) for j in range(y) for k in range(x)]
                at += max(f, y, x)
        out += rows[:a]
    return [list(p) for p in zip(*out)][:case["axes"]]


def _axis_of_pairs(case):
    """Which axis turns each pair: stretches of pairs one after the other (time a quarter, the
    others even parts of the rest), or the axes taking turns."""
    pairs, n = case["rot"] // 2, case["axes"]
    if case["mixed"]:
        return [i % n for i in range(pairs)]
    first = pairs if n == 1 else pairs // 4
    return [0 if i < first else 1 + (i - first) * (n - 1) // (pairs - first) for i in range(pairs)]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cu(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return _ints(out)


# ---------------------------------------------------------------- inputs

def _cached(normal, pages, hkv, page, d, top):
    """Pages and scales as a cache holds them: heads and channels of unlike size, some channels
    far larger than the others, quantised by blocks."""
    codes = torch.empty(pages, hkv, page, d, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, hkv, page // BLOCK, dtype=torch.uint8, device=DEV)
    size = torch.exp(0.4 * normal(1, hkv, 1, d)) * torch.where(normal(1, hkv, 1, d) > 2.3, 6.0, 1.0)
    for at in range(0, pages, 4096):  # (a part at a time, for its memory)
        x = normal(min(4096, pages - at), hkv, page, d) * size
        x = x.clamp(-top, top).unflatten(2, (page // BLOCK, BLOCK))
        e = _exponent(x.abs().amax((-2, -1)))
        codes[at:at + 4096] = _codes(x, e[..., None, None]).flatten(2, 3).view(torch.uint8)
        scales[at:at + 4096] = e.to(torch.uint8)
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + case["mix"])
    t = TYPES[case["type"]]
    h, hkv, d, page = case["h"], case["hkv"], case["d"], case["page"]
    new, full = _lengths(case)
    T, n = sum(new), case["n"]
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    s = dict(case=case, n=n, T=T, cu=_cu(new), kv_lens=_ints(full), places=None, axis=None)
    if case["op"] != "attend8":
        s["qkv"] = normal(T, (h + 2 * hkv) * d).to(t)
        s["qw"], s["kw"] = 1.0 + 0.3 * normal(d), 1.0 + 0.3 * normal(d)
        i = torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64)
        s["inv_freq"] = (1e6 ** (-2.0 * i / case["rot"])).float()
        if case["axes"]:
            s["places"], s["axis"] = _ints(_places(case)), _ints(_axis_of_pairs(case))
        s["q"] = torch.empty(T, h, d, dtype=t, device=DEV)
    if page == 0:
        s["k"] = torch.empty(T, hkv, d, dtype=t, device=DEV)
    else:
        shared = case.get("shared", 0) // page
        cols = -(-max(full) // page)
        used = [-(-x // page) - shared for x in full]
        pages = shared + sum(used) + 3
        order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32).tolist()
        table, at = [], shared
        for u in used:  # the shared pages first, then the sequence's own
            table.append(order[:shared] + order[at:at + u] + [0] * (cols - shared - u))
            at += u
        s["table"], s["pages"] = _ints(table), pages
        if case["op"] == "axes":
            s["kp"], s["vp"] = (normal(pages, hkv, page, d).to(t) for _ in range(2))
        else:
            top = TOP[case["type"]]
            (s["kp"], s["ks"]), (s["vp"], s["vs"]) = (_cached(normal, pages, hkv, page, d, top)
                                                      for _ in range(2))
    if case["op"] == "attend8":
        s["q"] = normal(T, h, d).to(t)
        s["shared"] = _ints([case["shared"]])
        s["o"] = torch.zeros(T, h, d, dtype=t, device=DEV)
    if own:
        import chunked_gated_delta_rule_amd as gdn
        s["gdn"] = gdn
        s["cfg"] = gdn.make_attn_config(
            T, n, h, hkv, d, dtype=t, rot_dim=case.get("rot", 0),
            rot_interleaved=case.get("inter", False), eps=EPS, page_size=page or 16,
            n_pages=s.get("pages", 0), max_pages=s["table"].shape[1] if "table" in s else 0,
            shared_max=case.get("shared", 0))
        if case["op"] == "attend8":
            s["ws"] = torch.empty(gdn.gdn_attn_paged8_workspace_size(s["cfg"]), dtype=torch.uint8,
                                  device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(s):
    gdn, op = s["gdn"], s["case"]["op"]
    if op == "attend8":
        gdn.gdn_attn_paged8(s["cfg"], s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["cu"], s["kv_lens"],
                            s["table"], s["shared"], s["o"], s["ws"])
        return {"o": s["o"]}
    if op == "append8":
        gdn.gdn_kv_append8(s["cfg"], s["qkv"], s["qw"], s["kw"], s["inv_freq"], s["places"], s["axis"],
                           s["cu"], s["kv_lens"], s["table"], s["q"], None, s["kp"], s["vp"], s["ks"],
                           s["vs"])
        return {n: s[n] for n in ("q", "kp", "vp", "ks", "vs")}
    if s["case"]["page"]:
        gdn.gdn_kv_append_axes(s["cfg"], s["qkv"], s["qw"], s["kw"], s["inv_freq"], s["places"],
                               s["axis"], s["cu"], s["kv_lens"], s["table"], s["q"], None, s["kp"],
                               s["vp"])
        return {n: s[n] for n in ("q", "kp", "vp")}
    gdn.gdn_qk_norm_rope_axes(s["cfg"], s["qkv"], s["qw"], s["kw"], s["inv_freq"], s["places"],
                              s["axis"], s["cu"], s["q"], s["k"])
    return {"q": s["q"], "k": s["k"]}


def _rows(s):
    """Sequence and place in the sequence's keys of every new token."""
    t = torch.arange(s["T"], device=DEV)
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return seq, s["kv_lens"].long()[seq] - s["cu"].long()[seq + 1] + t


def _norm_rope_rows(x, w, angle, inter):
    """Rows [T, heads, d] in 32 bits: RMS norm, weight, rotation of the first dims."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    half = angle.shape[-1]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :half], r[..., half:])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _plain_front(s):
    """q, k and v in 32 bits, and where their tokens belong."""
    c = s["case"]
    h, hkv, d = c["h"], c["hkv"], c["d"]
    seq, place = _rows(s)
    at = place.double()[:, None] if s["places"] is None else s["places"].double()[s["axis"].long()].T
    angle = at * s["inv_freq"].double()
    x = s["qkv"].float().view(s["T"], h + 2 * hkv, d)
    q = _norm_rope_rows(x[:, :h], s["qw"], angle, c["inter"])
    k = _norm_rope_rows(x[:, h:h + hkv], s["kw"], angle, c["inter"])
    return q, k, x[:, h + hkv:], seq, place


def _plain_axes(s):
    q, k, v, seq, place = _plain_front(s)
    t, page = s["qkv"].dtype, s["case"]["page"]
    if not page:
        return {"q": q.to(t), "k": k.to(t)}
    slot = s["table"].long()[seq, place // page]
    s["kp"][slot, :, place % page] = k.to(t)
    s["vp"][slot, :, place % page] = v.to(t)
    return {"q": q.to(t), "kp": s["kp"], "vp": s["vp"]}


def _exponent(a):
    """e of the least power of two 2^(e - 127) with a <= 448 times it (e4m3 ends at 448, which
    is 7/8 of 2^9), at least 2^-112."""
    m, x = torch.frexp(a)
    return (x - 9 + (m > 0.875) + 127).clamp(15, 247)


def _codes(x, e):
    return (x * torch.exp2(127.0 - e)).to(torch.float8_e4m3fn)


def _plain_append8(s):
    c = s["case"]
    q, k, v, seq, place = _plain_front(s)
    page, top = c["page"], TOP[c["type"]]
    slot, sub, row = s["table"].long()[seq, place // page], place % page // BLOCK, place % BLOCK
    # the blocks that the tokens lie in, each named by its first new token
    first = s["kv_lens"].long()[seq] - (s["cu"].long()[seq + 1] - s["cu"].long()[seq])
    lead = (row == 0) | (place == first)
    block = lead.long().cumsum(0) - 1
    slot_b, sub_b, had = slot[lead], sub[lead], row[lead]
    for name, x in (("k", k), ("v", v)):
        x = x.clamp(-top, top)
        codes, scales = s[name + "p"].view(torch.uint8), s[name + "s"].view(torch.uint8)
        a = torch.zeros(len(slot_b), c["hkv"], device=DEV)
        a.scatter_reduce_(0, block[:, None].expand(-1, c["hkv"]), x.abs().amax(-1), "amax")
        old = scales[slot_b, :, sub_b].int()
        e = torch.where(had[:, None] > 0, torch.maximum(old, _exponent(a)), _exponent(a))
        # the rows that the blocks had, by the new scales
        blocks = codes.unflatten(2, (page // BLOCK, BLOCK))
        rows = blocks[slot_b, :, sub_b].view(torch.float8_e4m3fn).float()
        again = (rows * torch.exp2((old - e).clamp(min=-126).float())[..., None, None])
        kept = torch.arange(BLOCK, device=DEV)[None, None, :, None] < had[:, None, None, None]
        blocks[slot_b, :, sub_b] = torch.where(kept, again, rows).to(torch.float8_e4m3fn).view(torch.uint8)
        blocks[slot, :, sub, row] = _codes(x, e[block][..., None]).view(torch.uint8)
        scales[slot_b, :, sub_b] = e.to(torch.uint8)
    return {"q": q.to(s["qkv"].dtype), **{n: s[n] for n in ("kp", "vp", "ks", "vs")}}


def _attend(q, k, v, last, scale):
    """q [n, hkv, rows, d]; k, v [n, hkv, keys, d] in 32 bits; last [n, rows]: the
    last key that each row sees (-1: none, and its output is zero)."""
    key = torch.arange(k.shape[2], device=DEV)
    seen = (key <= last[..., None])[:, None]
    p = torch.matmul(q, k.transpose(2, 3)).mul_(scale).masked_fill_(~seen, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def _read(s, name):
    """The cache's numbers at every position of the table: [n, hkv, keys, d] in 32 bits."""
    c, at = s["case"], s["table"].long()
    x = s[name + "p"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    e = s[name + "s"].view(torch.uint8)[at].view(torch.float8_e8m0fnu).float()
    x = x.unflatten(3, (c["page"] // BLOCK, BLOCK)).mul_(e[..., None, None])
    return x.permute(0, 2, 1, 3, 4, 5).reshape(s["n"], c["hkv"], -1, c["d"])


def _plain_attend8(s):
    c = s["case"]
    h, hkv, d, n, most = c["h"], c["hkv"], c["d"], s["n"], c["tokens"] // c["n"]
    seq, place = _rows(s)
    g = h // hkv
    q = s["q"].float().view(n, most, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, most * g, d)
    o = _attend(q, _read(s, "k"), _read(s, "v"), place.view(n, most).repeat_interleave(g, 1),
                1.0 / math.sqrt(d))
    return {"o": o.view(n, hkv, most, g, d).permute(0, 2, 1, 3, 4).reshape(s["T"], h, d).to(s["q"].dtype)}


_PLAIN = {"axes": _plain_axes, "append8": _plain_append8, "attend8": _plain_attend8}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    new, full = _lengths(case)
    T, h, hkv, d = sum(new), case["h"], case["hkv"], case["d"]
    places = 4 * T * case.get("axes", 0)
    if case["op"] == "axes":
        heads = h + (2 if case["page"] else 1) * hkv
        return {"bytes": 2 * d * T * 2 * heads + places, "flops": 9 * d * T * (h + hkv)}
    if case["op"] == "append8":
        return {"bytes": d * T * (2 * (h + 2 * hkv) + 2 * h + 2 * hkv) + places,
                "flops": 9 * d * T * (h + hkv) + 4 * d * T * hkv}
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(new, full))
    keys = sum(full)  # the pages that all sequences share are read once
    keys -= (case["n"] - 1) * (case["shared"] // case["page"] * case["page"])
    return {"bytes": d * (2 * 2 * T * h + 2 * keys * hkv) + keys * hkv // 8, "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _turned(x, w, turn, inter):
    """Unit root mean square, weight, and the pairs of dims as complex numbers turned."""
    x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS)
    x = x * w.double()
    r = 2 * turn.shape[-1]
    pair = x[..., :r].unflatten(-1, (r // 2, 2) if inter else (2, r // 2))
    pair = pair if inter else pair.transpose(-1, -2)
    pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
    pair = pair if inter else pair.transpose(-1, -2)
    return torch.cat((pair.flatten(-2), x[..., r:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attend8(s) if case["op"] == "attend8" else _exact_front(s)


def _exact_front(s):
    case = s["case"]
    new, full = _lengths(case)
    h, hkv, d, page = case["h"], case["hkv"], case["d"], case["page"]
    places = _places(case) if case["axes"] else None
    axis = _axis_of_pairs(case) if case["axes"] else None
    q, k = [], []
    state = {n: s[n].double() for n in ("kp", "vp", "ks", "vs") if n in s}
    begin = 0
    for i, (a, b) in enumerate(zip(new, full)):
        x = s["qkv"][begin:begin + a].double().reshape(a, h + 2 * hkv, d)
        at = torch.arange(b - a, b, device=DEV)
        if places:
            by = torch.tensor([p[begin:begin + a] for p in places], device=DEV).double()[axis].T
        else:
            by = at.double()[:, None]
        angle = by * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)
        begin += a
        q.append(_turned(x[:, :h], s["qw"], turn, case["inter"]))
        kk, vv = _turned(x[:, h:h + hkv], s["kw"], turn, case["inter"]), x[:, h + hkv:]
        k.append(kk)
        if page == 0:
            continue
        pages = s["table"][i].long()[at.div(page, rounding_mode="floor")]
        if case["op"] == "axes":
            state["kp"][pages, :, at % page], state["vp"][pages, :, at % page] = kk, vv
            continue
        for name, y in (("k", kk), ("v", vv)):
            y = y.clamp(-TOP[case["type"]], TOP[case["type"]])
            _exact_blocks(state[name + "p"], state[name + "s"], s["table"][i].long(), page, b - a, y)
    out = {"q": torch.cat(q), **state}
    return out if page else {"q": out["q"], "k": torch.cat(k)}


def _exact_blocks(pool, scales, table, page, at, y):
    """Writes the rows y of positions at, at + 1, ... in units of their blocks' scales."""
    had = at % BLOCK
    blocks = -(-(had + len(y)) // BLOCK)
    pad = torch.zeros(blocks * BLOCK, *y.shape[1:], dtype=torch.float64, device=DEV)
    pad[had:had + len(y)] = y
    pad = pad.unflatten(0, (blocks, BLOCK))
    place = at - had + BLOCK * torch.arange(blocks, device=DEV)
    where, sub = table[place.div(page, rounding_mode="floor")], place % page // BLOCK
    most = pad.abs().amax((1, 3))
    # the least whole E with most <= 448 2^E, at least -112
    E = torch.floor(torch.log2(most.clamp(min=1e-300) / 448)).clamp(min=-112)
    E = torch.where(most > 448 * 2.0 ** E, E + 1, E)
    scale = 2.0 ** E
    before = scales[where, :, sub]
    if had:
        scale[0] = torch.maximum(scale[0], before[0])
    rows = pool.unflatten(2, (page // BLOCK, BLOCK))
    for b in range(blocks):
        lo = had if b == 0 else 0
        hi = min(BLOCK, had + len(y) - b * BLOCK)
        rows[where[b], :, sub[b], :lo] *= (before[b] / scale[b])[:, None, None]
        rows[where[b], :, sub[b], lo:hi] = (pad[b, lo:hi] / scale[b][:, None]).transpose(0, 1)
    scales[where, :, sub] = scale


def _exact_attend8(s):
    case = s["case"]
    new, full = _lengths(case)
    h, hkv, d, page = case["h"], case["hkv"], case["d"], case["page"]
    out = torch.zeros(sum(new), h, d, dtype=torch.float64, device=DEV)
    begin = 0
    for i, (a, b) in enumerate(zip(new, full)):
        rows = s["table"][i, :-(-b // page)].long()
        k, v = ((s[n + "p"].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double() *
                 s[n + "s"].view(torch.uint8)[rows].view(torch.float8_e8m0fnu).double()
                 .repeat_interleave(BLOCK, 2)[..., None]).transpose(1, 2).reshape(-1, hkv, d)[:b]
                for n in ("k", "v"))
        for head in range(h):
            kk, vv = k[:, head * hkv // h], v[:, head * hkv // h]
            score = s["q"][begin:begin + a, head].double() @ kk.T * d ** -0.5
            score = score + torch.full_like(score, -math.inf).triu(b - a + 1)
            out[begin:begin + a, head] = torch.softmax(score, -1) @ vv
        begin += a
    return {"o": out}
