"""CPU pins of the softmax-attention oracle by closed forms, and planted mistakes
that the pins and the bounds catch."""

import math

import numpy as np
import pytest
import torch

import chunked_gated_delta_rule_amd as gdn
from attn_helpers import check_attention, check_norm_rope
from oracle import attention

RNG = np.random.Generator(np.random.PCG64(5))


def test_norm_gives_unit_root_mean_square():
    x = RNG.standard_normal((4, 3, 128)) * 37.0
    y, _ = attention.norm_rope(x, np.ones(128), np.zeros(4), None, 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    w = RNG.standard_normal(128)
    z, _ = attention.norm_rope(x, w, np.zeros(4), None, 0.0)
    assert np.allclose(z, y * w)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_by_hand(inter):
    """One pair a quarter turn, one half a turn, one not at all, the rest untouched."""
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    f = np.array([math.pi / 2, math.pi, 0.0])
    y, _ = attention.norm_rope(x, None, np.array([1.0]), f, 0.0, interleaved=inter)
    want = [-2, 1, -3, -4, 5, 6, 7, 8] if inter else [-4, -2, 3, 1, -5, 6, 7, 8]
    assert np.allclose(y[0, 0], want)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_makes_scores_depend_on_the_distance_alone(inter):
    q, k = RNG.standard_normal((2, 1, 1, 64))
    f = 10.0 ** -np.arange(32.0)
    at = lambda x, p: attention.norm_rope(x, None, np.array([p]), f, 0.0, inter)[0][0, 0]  # noqa: E731
    assert math.isclose(at(q, 900.0) @ at(k, 893.0), at(q, 7.0) @ at(k, 0.0), rel_tol=1e-9)


def test_attention_of_equal_keys_is_the_mean_of_what_is_seen():
    v = RNG.standard_normal((5, 1, 8))
    o, _, total = attention.attend(np.ones((5, 2, 8)), np.ones((5, 1, 8)), v, 0.3)
    for i in range(5):
        assert np.allclose(o[i], v[:i + 1, 0].mean(0))
        assert np.allclose(total[i], i + 1)


def test_attention_of_a_sharp_score_picks_the_key_and_rows_without_keys_are_zero():
    k = np.eye(6)[:, None] * 1000.0
    v = RNG.standard_normal((6, 1, 6))
    o, _, _ = attention.attend(np.eye(6)[:, None], k, v, 1.0)
    assert np.allclose(o, v)
    o, _, _ = attention.attend(np.ones((4, 1, 6)), k[:2], v[:2], 1.0)  # rows 0, 1 see nothing
    assert np.all(o[:2] == 0) and np.allclose(o[2], v[0])


def test_positions_and_gather():
    cu = np.array([0, 2, 2, 5])
    assert list(attention.positions(cu)) == [0, 1, 0, 1, 2]
    assert list(attention.positions(cu, [9, 4, 3])) == [7, 8, 0, 1, 2]
    pages = np.arange(3 * 2 * 4 * 1.0).reshape(3, 2, 4, 1)
    rows = attention.gather(pages, [2, 0], 6)
    assert list(rows[:, 1, 0]) == [20, 21, 22, 23, 4, 5]


def test_scaled_frequencies():
    f = gdn.rope_inv_freq(64, base=1e6)
    assert f.dtype == torch.float32 and f[0] == 1.0
    assert torch.allclose(f[1:] / f[:-1], torch.full((31,), 1e6 ** (-1 / 32)))
    assert torch.allclose(gdn.rope_inv_freq(64, 1e6, factor=8.0), f / 8)
    g = gdn.rope_inv_freq(64, 1e6, factor=8.0, original_len=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32])
    assert torch.allclose(g[turns <= 1], f[turns <= 1] / 8)
    assert ((g <= f * 1.000001) & (g >= f / 8 * 0.999999)).all() and (turns <= 1).any()
    assert gdn.rope_inv_freq(0).numel() == 0
    for bad in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=4, factor=0.0),
                dict(rot_dim=4, base=-1.0), dict(rot_dim=4, original_len=8, low_turns=4, high_turns=4)):
        with pytest.raises(ValueError):
            gdn.rope_inv_freq(**bad)


def _attention_case(t):
    q, k, v = (torch.from_numpy(RNG.standard_normal(s)).to(t).double().numpy()
               for s in ((9, 2, 128), (13, 1, 128), (13, 1, 128)))
    return q, k, v, 128 ** -0.5


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_the_bounds_pass_a_rounded_result_and_catch_planted_mistakes(t):
    q, k, v, scale = _attention_case(t)
    o, _, _ = attention.attend(q, k, v, scale)
    check_attention(torch.from_numpy(o).to(t), q, k, v, scale, t)
    off_by_one = attention.attend(q, k[:12], v[:12], scale)[0]
    no_scale = attention.attend(q, k, v, 1.0)[0]
    other_head = attention.attend(q[:, ::-1], k, v, scale)[0]
    for wrong in (off_by_one, no_scale, other_head, o * (1 + 4 * torch.finfo(t).eps)):
        with pytest.raises(AssertionError):
            check_attention(torch.from_numpy(np.ascontiguousarray(wrong)).to(t), q, k, v, scale, t)


def test_the_bounds_catch_mistakes_in_norm_and_rotation():
    t = torch.float16
    x = torch.from_numpy(RNG.standard_normal((3, 2, 128))).to(t).double().numpy()
    w, p, f = np.ones(128), np.array([5.0, 6, 7]), 1e4 ** -np.arange(0, 1, 1 / 32)
    y, mag = attention.norm_rope(x, w, p, f, 1e-6)
    check_norm_rope(torch.from_numpy(y).to(t), y, mag, t)
    for wrong in (attention.norm_rope(x, w, p + 1, f, 1e-6)[0],
                  attention.norm_rope(x, w, -p, f, 1e-6)[0],
                  attention.norm_rope(x, w, p, f, 1e-6, True)[0],
                  attention.norm_rope(x, None, p, f, 1e-6)[0],
                  attention.norm_rope(x, w, p, f, 1e-6, rot_scale=1.01)[0]):
        with pytest.raises(AssertionError):
            check_norm_rope(torch.from_numpy(wrong).to(t), y, mag, t)
