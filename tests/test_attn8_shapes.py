"""The tests' account of how the append to an 8-bit cache is cut: its numbering of blocks and
parts, and the shapes that the GPU tests mean to reach."""

import random

import pytest

import attn8_shapes
import chunked_gated_delta_rule_amd as gdn


def cfg(tokens, n=1, h=16, hkv=2, d=256):
    return gdn.make_attn_config(tokens, n, h, hkv, d)


@pytest.mark.parametrize("seed", range(3))
def test_every_part_of_every_slot_has_one_work_group(seed):
    rng = random.Random(seed)
    kinds = set()
    for _ in range(60):
        hkv = rng.choice([1, 2, 8])
        s = attn8_shapes.append8(cfg(int(2 ** rng.uniform(0, 15.5)), rng.choice([1, 3, 40, 300]),
                                     hkv * rng.choice([1, 4, 8]), hkv), 256)
        assert s.slots % s.group == 0
        at = attn8_shapes.places(s)
        assert len(set(at)) == s.slots * s.parts == len(at)
        assert all(0 <= a < s.slots and 0 <= b < s.parts for a, b in at)
        kinds.add((s.whole, s.parts > 1))
    assert len(kinds) >= 3


@pytest.mark.parametrize("seed", range(20))
def test_blocks_have_slots_of_their_own(seed):
    """Any lengths (none among them) and first positions, below zero too."""
    rng = random.Random(seed)
    lens = [rng.choice([0, 1, 2, 15, 16, 17, 18, 31, 33, rng.randrange(200)]) for _ in range(rng.randrange(1, 40))]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    at = attn8_shapes.slots_of(cu, [rng.randrange(-40, 400) for _ in lens])
    assert all(a < b for a, b in zip(at, at[1:]))
    room = attn8_shapes.append8(cfg(max(cu[-1], 1), len(lens)), 256).slots
    assert not at or at[-1] < room


@pytest.mark.parametrize("tokens,n,h,hkv,d,parts,whole,past", [
    (32768, 4, 16, 2, 256, 3, False, True), (30004, 3, 32, 4, 128, 4, False, True),
    (24001, 2, 16, 2, 128, 3, False, False), (40000, 4, 2, 2, 128, 1, True, False),
    (2500, 40, 32, 4, 128, 6, True, False), (256, 256, 32, 8, 128, 1, True, False)])
def test_shapes(tokens, n, h, hkv, d, parts, whole, past):
    s = attn8_shapes.append8(cfg(tokens, n, h, hkv, d), 256)
    assert (s.parts, s.whole, s.past_cache) == (parts, whole, past)
