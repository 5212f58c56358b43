"""How a call of gdn_kv_append8 is cut (launch_attn_append8 in csrc/attn_append8.hip over
again, its thresholds read from the sources), for tests that mean to reach one launch shape."""

import os
import re
from types import SimpleNamespace

from attn_shapes import CSRC


def _number(file, name):
    text = open(os.path.join(CSRC, file)).read()
    value = re.search(r"\b%s = ([0-9 <]+)[;,]" % name, text).group(1)
    base, _, shift = value.partition("<<")
    return int(base) << int(shift or 0)


BLOCK = _number("attn_append8.hip", "kBlock")
LEAST = _number("attn_append8.hip", "kLeastPasses")
MOST = _number("attn_append8.hip", "kMostPasses")
PAST = _number("attn_common.hpp", "kPastCache")


def append8(c, cus, q=True, k=True):
    """parts: work-groups per block of tokens; group: blocks that are numbered together;
    whole: all of them at once; past_cache: q and k are stored past the caches."""
    each = -(-c.t_max // c.n_max)
    blocks = c.n_max * -(-each // BLOCK)
    passes = -(-min(each, BLOCK) * (c.h + 2 * c.hkv) // BLOCK)
    least = min(max(blocks * passes // (4 * cus), LEAST), MOST)
    parts = max(min(32 * cus // blocks, passes // least), 1)
    slots = -(-(c.t_max // BLOCK + 2 * c.n_max) // 8) * 8
    whole = slots * parts <= 16 * cus
    heads = (c.h if q else 0) + (c.hkv if k else 0) + c.hkv
    return SimpleNamespace(parts=parts, slots=slots, whole=whole, group=slots if whole else 8,
                           past_cache=heads * c.t_max * c.d * 2 > PAST)


def places(s):
    """(slot, part) of every work-group in the order of their numbers."""
    out = []
    for wg in range(s.slots * s.parts):
        group, at = divmod(wg, s.group * s.parts)
        out.append((s.group * group + at % s.group, (at // s.group + group) % s.parts))
    return out


def slots_of(cu, pos0):
    """Slots of the blocks of 16 positions that a batch's tokens lie in, in order; pos0: each
    sequence's first new position."""
    out = []
    for s, p in enumerate(pos0):
        n = cu[s + 1] - cu[s]
        blocks = (p + n - 1) // BLOCK - p // BLOCK + 1 if n else 0
        out += [cu[s] // BLOCK + 2 * s + i for i in range(blocks)]
    return out
