"""CPU pins of the oracle of the 8-bit cache and of rotations by several axes, by closed
forms and by torch's own float8 types, and planted mistakes that the checks catch."""

import math

import numpy as np
import pytest
import torch

import chunked_gated_delta_rule_amd as gdn
from attn8_helpers import Cache8, check_codes, quantised
from oracle import attention, cache8

RNG = np.random.Generator(np.random.PCG64(6))


def test_every_code_has_its_value():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache8.VALUES, want, equal_nan=True)
    scales = torch.arange(256, dtype=torch.uint8).view(torch.float8_e8m0fnu).double().numpy()
    assert np.array_equal(cache8.scale_value(np.arange(256)), scales, equal_nan=True)


def test_encoding_is_the_nearest_code_and_ties_are_even():
    mid = (cache8.GRID[:-1] + cache8.GRID[1:]) / 2
    x = np.concatenate([cache8.GRID, mid, mid * (1 + 1e-12), mid * (1 - 1e-12),
                        RNG.standard_normal(4000) * 100])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # (torch rounds to fp32 first: the neighbours of a tie are put beside it by hand)
    near = np.isin(np.abs(x), mid * (1 + 1e-12)) | np.isin(np.abs(x), mid * (1 - 1e-12))
    got = cache8.encode(x)
    assert np.array_equal(got[~near], want[~near])
    n = len(cache8.GRID) - 1
    at = len(cache8.GRID) + n
    assert np.array_equal(got[at:at + n], np.arange(1, n + 1))
    assert np.array_equal(got[at + n:at + 2 * n], np.arange(n))
    assert cache8.encode(np.array([np.nan]))[0] == 127


@pytest.mark.parametrize("a,e", [(0.0, 15), (448.0, 127), (448.0001, 128), (449.0, 128), (224.0, 126),
                                 (223.9, 126), (1.0, 119), (1.75, 119), (1.7500001, 120), (61440.0, 135),
                                 (1.875 * 2.0 ** 127, 247), (2.0 ** -120, 15)])
def test_least_scale(a, e):
    assert cache8.least_scale(a) == e
    assert a <= 448.0 * 2.0 ** (e - 127) and (e == 15 or a > 448.0 * 2.0 ** (e - 128))


def test_appending_grows_a_blocks_scale_and_rounds_its_rows_again():
    codes = np.full((2, 1, 16, 4), 0x7f, np.uint8)
    scales = np.full((2, 1, 1), 200, np.uint8)
    row = np.array([1, 0], np.int32)
    one = lambda v: np.full((1, 1, 4), v)  # noqa: E731
    cache8.append(codes, scales, row, 0, one(0.4375), 1e30)   # 448 2^-10: e = 117
    assert scales[1, 0, 0] == 117 and np.all(codes[1, 0, 0] == cache8.encode(np.array(448.0)))
    cache8.append(codes, scales, row, 1, one(-0.001), 1e30)   # fits
    assert scales[1, 0, 0] == 117
    before = cache8.values(codes, scales)[1, 0, 1, 0]
    cache8.append(codes, scales, row, 2, one(7.0), 1e30)      # 448 2^-6: e = 121
    assert scales[1, 0, 0] == 121
    got = cache8.values(codes, scales)[1, 0, :3, 0]
    assert got[0] == 0.4375 and got[2] == 7.0
    assert abs(got[1] - before) <= 2.0 ** -10 * 2.0 ** -6     # half a subnormal step
    cache8.append(codes, scales, row, 16, one(3.0), 1e30)     # the next page's block begins anew
    assert scales[0, 0, 0] == cache8.least_scale(3.0)
    cache8.append(codes, scales, row, 0, one(1e-3), 1e30)     # and so does one written again
    assert scales[1, 0, 0] == cache8.least_scale(1e-3)


def test_values_that_are_not_finite_and_the_top():
    codes, scales = np.zeros((1, 1, 16, 4), np.uint8), np.zeros((1, 1, 1), np.uint8)
    x = np.array([[[np.nan, np.inf, 65504.0, -1.0]]])
    cache8.append(codes, scales, np.array([0]), 3, x, cache8.TOP["float16"])
    got = cache8.values(codes, scales)[0, 0, 3]
    assert np.isnan(got[0]) and np.isnan(got[1]) and got[2] == 61440.0 and np.isfinite(got[3])


def test_one_axis_is_the_plain_rotation():
    x, w = RNG.standard_normal((5, 2, 64)), RNG.standard_normal(64)
    f = 10.0 ** -np.arange(16.0)
    pos = np.arange(5.0) * 7
    for inter in (False, True):
        a = attention.norm_rope(x, w, pos, f, 1e-6, inter, 1.5)
        b = cache8.norm_rope_axes(x, w, [pos * 3, pos], np.ones(16), f, 1e-6, inter, 1.5)
        assert np.allclose(a[0], b[0], rtol=0, atol=1e-12) and np.allclose(a[1], b[1])


def test_each_pair_turns_by_its_axis():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    f = np.array([math.pi / 2] * 3)
    y, _ = cache8.norm_rope_axes(x, None, [[0.0], [1.0], [2.0]], [0, 1, 2], f, 0.0)
    assert np.allclose(y[0, 0], [1, -5, -3, 4, 2, -6])


def test_planted_mistakes_are_caught():
    x = RNG.standard_normal((3, 1, 16, 32))
    codes, scales = quantised(x, 1e30)
    mag = np.abs(x)
    check_codes(codes, scales[:, :, 0][..., None].repeat(16, 2), x, mag)
    wrong = codes.copy()
    wrong[1, 0, 5, 7] ^= 1
    with pytest.raises(AssertionError):
        check_codes(wrong, scales[:, :, 0][..., None].repeat(16, 2), x, mag)
    with pytest.raises(AssertionError):
        check_codes(codes, scales[:, :, 0][..., None].repeat(16, 2) + 1, x, mag)


def test_the_pool_of_the_tests_is_what_it_says():
    c = Cache8([33, 0, 5], 2, 32, 16, torch.bfloat16, 3)
    for s, n in enumerate(c.lens):
        k, v = c.rows(s)
        assert k.shape == (n, 2, 32) and np.isfinite(k).all() and np.isfinite(v).all()
    assert np.isnan(cache8.values(c.k, c.ks)[c.table[0, 2], :, 1:]).all()


@pytest.mark.parametrize("sections,inter,want", [
    ((2, 1, 1), False, [0, 0, 1, 2]), ((2, 1, 1), True, [0, 1, 2, 0]), ((3,), True, [0, 0, 0]),
    ((1, 3), True, [0, 1, 1, 1]), ((0, 2), False, [1, 1]), ((0, 1, 0, 2), True, [1, 3, 3])])
def test_rope_pair_axis(sections, inter, want):
    assert gdn.rope_pair_axis(sections, inter).tolist() == want


def test_rope_pair_axis_refuses():
    for bad in ((), (1, -1)):
        with pytest.raises(ValueError, match="sections"):
            gdn.rope_pair_axis(bad)


def test_a_growing_scale_moves_a_row_by_half_its_smallest_step():
    """Rows of a block, then others of any size: each growth to e moves what is there by
    2^(e - 137) at most, which is below 2^-17 of the value that asked for it; and a block that
    is put back and appended to again is what it would have been."""
    moved = 0
    for seed in range(8):
        rng = np.random.Generator(np.random.PCG64(seed))
        codes, scales = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1, 1), np.uint8)
        top, at = 1.875 * 2.0 ** 127, 0
        while at < 15:
            n = min(int(rng.integers(1, 4)), 16 - at)
            x = rng.standard_normal((n, 1, 64)) * 2.0 ** rng.integers(-4, 12)
            was, old = cache8.values(codes, scales)[0, 0, :at], scales.copy()
            kept = codes.copy()
            cache8.append(codes, scales, [0], at, x, top)
            off, e = np.abs(cache8.values(codes, scales)[0, 0, :at] - was), int(scales[0, 0, 0])
            if at and e > old[0, 0, 0]:
                assert np.all(off <= 2.0 ** (e - 137)) and 2.0 ** (e - 137) < 2.0 ** -17 * np.abs(x).max()
                moved += np.any(off > 0)
            else:
                assert not off.any()
            cache8.append(kept, old, [0], at, x, top)
            assert np.array_equal(kept, codes) and np.array_equal(old, scales)
            at += n
    assert moved
