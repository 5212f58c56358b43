"""Host-side checks of the 8-bit cache's entry points and of the rotations by several
axes: every bad argument is refused with the documented status before any HIP call, and the
binding refuses tensors that do not fit. No test here launches a kernel."""

import ctypes

import pytest
import torch

import chunked_gated_delta_rule_amd as gdn
from test_attn_host import FRONT, INVALID, OK, P, UNSUPPORTED, WORKSPACE, cfg, refused

AXES = {**{k: v for k, v in FRONT.items() if k != "kv_lens"}}
CACHE = dict(block_table=P, k_pages=P, v_pages=P)
SCALES = dict(k_scales=P, v_scales=P)


def status_of(name, c, args, n_axes=3, positions=P, pair_axis=P):
    """The C call itself (the binding takes positions as tensors)."""
    a = dict(args)
    head = [ctypes.byref(c), a.pop("qkv"), 0, a.pop("q_w"), a.pop("k_w"), a.pop("inv_freq"), positions,
            pair_axis, n_axes]
    order = ["cu_seqlens", "kv_lens", "block_table", "q", "k", "k_pages", "v_pages", "k_scales", "v_scales"]
    rest = [a[k] for k in order if k in a]
    return getattr(gdn.load_library(), name)(*head, *rest, None)


NAMES = {"gdn_qk_norm_rope_axes": AXES, "gdn_kv_append_axes": {**FRONT, **CACHE},
         "gdn_kv_append8": {**FRONT, **CACHE, **SCALES}}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(cu_seqlens=None), dict(kv_lens=None), dict(block_table=None),
    dict(k_pages=None), dict(v_pages=None), dict(k_scales=None), dict(v_scales=None),
    dict(inv_freq=None), dict(qkv=P + 8), dict(q=P + 8), dict(k=P + 8), dict(k_pages=P + 8),
    dict(v_pages=P + 4), dict(q_w=P + 1), dict(k_w=P + 2), dict(inv_freq=P + 3),
    dict(cu_seqlens=P + 2), dict(kv_lens=P + 1), dict(block_table=P + 2)])
def test_front_refusals(name, change):
    args = NAMES[name]
    if not set(change) <= set(args):
        return
    assert status_of(name, cfg(), {**args, **change}) == INVALID


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("change", [
    dict(positions=None), dict(pair_axis=None), dict(n_axes=0), dict(n_axes=-1),
    dict(n_axes=gdn.GDN_AXES_LIMIT + 1), dict(positions=P + 2), dict(pair_axis=P + 1)])
def test_axes_refusals(name, change):
    assert status_of(name, cfg(), NAMES[name], **change) == INVALID


def test_axes_need_a_rotation_and_q_and_k_are_required_without_a_cache():
    c = cfg(rot_dim=0)
    for name, args in NAMES.items():
        assert status_of(name, c, {**args, "inv_freq": None}) == INVALID
    for missing in ("q", "k"):
        assert status_of("gdn_qk_norm_rope_axes", cfg(), {**AXES, missing: None}) == INVALID
    # one axis: none of the three
    assert status_of("gdn_kv_append8", cfg(t_max=0), NAMES["gdn_kv_append8"], 0, None, None) == OK
    for name in ("gdn_qk_norm_rope_axes", "gdn_kv_append_axes"):
        assert status_of(name, cfg(t_max=0), NAMES[name], 0, None, None) == INVALID


@pytest.mark.parametrize("field", ["n_pages", "max_pages"])
def test_cache_calls_need_pages(field):
    for name in ("gdn_kv_append_axes", "gdn_kv_append8"):
        assert status_of(name, cfg(**{field: 0}), NAMES[name]) == INVALID
    refused(INVALID, gdn.gdn_attn_paged8, cfg(**{field: 0}), **PAGED8)


@pytest.mark.parametrize("field,value,status", [
    ("d", 64, UNSUPPORTED), ("dtype", gdn.GDN_F32, UNSUPPORTED), ("h", 9, UNSUPPORTED),
    ("page_size", 8, UNSUPPORTED), ("rot_dim", 3, INVALID), ("eps", -1.0, INVALID)])
def test_configs_are_checked(field, value, status):
    c = cfg(**{field: value})
    for name, args in NAMES.items():
        assert status_of(name, c, args) == status
    out = ctypes.c_size_t(0)
    lib = gdn.load_library()
    assert lib.gdn_attn_paged8_workspace_size(ctypes.byref(c), ctypes.byref(out)) == status
    refused(status, gdn.gdn_attn_paged8, c, **PAGED8)


def test_workspace_size():
    lib, out = gdn.load_library(), ctypes.c_size_t(0)
    assert lib.gdn_attn_paged8_workspace_size(None, ctypes.byref(out)) == INVALID
    assert lib.gdn_attn_paged8_workspace_size(ctypes.byref(cfg()), None) == INVALID
    n = gdn.gdn_attn_paged8_workspace_size(cfg())
    assert n >= 256 and n % 256 == 0


PAGED8 = dict(q=P, k_pages=P, v_pages=P, k_scales=P, v_scales=P, cu_seqlens=P, kv_lens=P, block_table=P,
              shared_len=None, o=P, workspace=P, ws_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID),
    (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID), (dict(cu_seqlens=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(block_table=None), INVALID), (dict(o=None), INVALID),
    (dict(q=P + 8), INVALID), (dict(k_pages=P + 8), INVALID), (dict(v_pages=P + 1), INVALID),
    (dict(o=P + 2), INVALID), (dict(shared_len=P + 2), INVALID), (dict(kv_lens=P + 2), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=P + 64), WORKSPACE),
    (dict(ws_bytes=255), WORKSPACE),
])
def test_paged8_refusals(change, status):
    refused(status, gdn.gdn_attn_paged8, cfg(), **{**PAGED8, **change})


@pytest.mark.parametrize("row", [8 * 128 - 8, 8 * 128 + 4, -8, (1 << 24) + 8])
def test_row_strides_are_checked(row):
    lib, b = gdn.load_library(), ctypes.byref(cfg())
    assert lib.gdn_attn_paged8(b, P, row, P, P, P, P, P, P, P, None, P, P, 1 << 40, None) == INVALID
    assert lib.gdn_qk_norm_rope_axes(b, P, row, P, P, P, P, P, 3, P, P, P, None) == INVALID
    assert lib.gdn_kv_append8(b, P, row, P, P, P, P, P, 3, P, P, P, P, P, P, P, P, P, None) == INVALID


def test_nothing_to_do_is_fine_without_a_device():
    c = cfg(t_max=0)
    for name, args in NAMES.items():
        assert status_of(name, c, args) == OK
    gdn.gdn_attn_paged8(c, **PAGED8, stream=0)


def test_binding_refuses_tensors_that_do_not_fit():
    """Host tensors stand in: every check but the last one (device) comes first."""
    c, t, i32 = cfg(), torch.bfloat16, torch.int32
    codes, scales = torch.zeros(9, 2, 16, 128, dtype=torch.uint8), torch.zeros(9, 2, 1, dtype=torch.uint8)
    good = dict(q=torch.zeros(64, 8, 128, dtype=t), k_pages=codes, v_pages=codes.view(torch.float8_e4m3fn),
                k_scales=scales, v_scales=scales.view(torch.float8_e8m0fnu),
                cu_seqlens=torch.zeros(5, dtype=i32), kv_lens=torch.zeros(4, dtype=i32),
                block_table=torch.zeros(4, 3, dtype=i32), shared_len=None,
                o=torch.zeros(64, 8, 128, dtype=t), workspace=P, ws_bytes=1 << 40)

    def bad(match, **change):
        with pytest.raises(ValueError, match=match):
            gdn.gdn_attn_paged8(c, **{**good, **change}, stream=0)

    bad("device tensor")
    bad("k_pages: dtype", k_pages=codes.to(t))
    bad("v_pages: dtype", v_pages=codes.view(torch.float8_e5m2))
    bad("k_scales: dtype", k_scales=scales.float())
    bad("v_scales: dtype", v_scales=scales.view(torch.float8_e4m3fn))
    bad("k_pages: .* elements", k_pages=codes[:8])
    bad("v_scales: .* elements", v_scales=scales[:8])
    bad("last dimension", k_scales=torch.zeros(9, 2, 2, dtype=torch.uint8))
    bad("contiguous", k_pages=torch.zeros(9, 2, 16, 256, dtype=torch.uint8)[..., ::2])
    qkv, pos, axis = torch.zeros(64, 12 * 128, dtype=t), torch.zeros(3, 64, dtype=i32), torch.zeros(32, dtype=i32)
    front = dict(qkv=qkv, q_w=None, k_w=None, inv_freq=torch.zeros(32), cu_seqlens=good["cu_seqlens"],
                 q=good["q"], k=torch.zeros(64, 2, 128, dtype=t))

    def bad_axes(match, positions=pos, pair_axis=axis):
        with pytest.raises(ValueError, match=match):
            gdn.gdn_qk_norm_rope_axes(c, **front, positions=positions, pair_axis=pair_axis, stream=0)

    bad_axes("device tensor")
    bad_axes("positions", positions=pos[:, :63])
    bad_axes("positions", positions=pos[0])
    bad_axes("positions", positions=None)
    bad_axes("pair_axis", pair_axis=None)
    bad_axes("pair_axis", pair_axis=P)
    bad_axes("dtype", positions=pos.long())
    bad_axes("pair_axis: 31", pair_axis=axis[:31])
    bad_axes("contiguous", positions=torch.zeros(64, 3, dtype=i32).t())


def test_high_level_calls_refuse_and_take_no_tokens():
    t, i32 = torch.bfloat16, torch.int32
    cu, kv = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    codes, scales = torch.zeros(3, 2, 32, 128, dtype=torch.uint8), torch.zeros(3, 2, 2, dtype=torch.uint8)
    table = torch.zeros(2, 2, dtype=i32)
    qkv, q = torch.zeros(4, 8 * 128, dtype=t), torch.zeros(4, 4, 128, dtype=t)
    for one in (dict(k_scales=scales), dict(v_scales=scales)):
        with pytest.raises(ValueError, match="go together"):
            gdn.append_paged_kv(qkv, 4, cu, kv, table, codes, codes, **one)
        with pytest.raises(ValueError, match="go together"):
            gdn.paged_attention(q, codes, codes, cu, kv, table, **one)
    pos, axis = torch.zeros(3, 4, dtype=i32), torch.zeros(32, dtype=i32)
    with pytest.raises(ValueError, match="kv_lens"):
        gdn.qk_norm_rope(qkv, 4, 2, cu, inv_freq=torch.zeros(32), kv_lens=kv, positions=pos, pair_axis=axis)
    with pytest.raises(ValueError, match="pair_axis"):
        gdn.qk_norm_rope(qkv, 4, 2, cu, inv_freq=torch.zeros(32), positions=pos)
    empty = gdn.append_paged_kv(qkv[:0], 4, cu, kv, table, codes, codes.clone(), k_scales=scales,
                                v_scales=scales.clone(), output_k=True)
    assert empty[0].shape == (0, 4, 128) and empty[1].shape == (0, 2, 128)
    assert gdn.paged_attention(q[:0], codes, codes, cu, kv, table, k_scales=scales,
                               v_scales=scales).shape == (0, 4, 128)
    a, b = gdn.qk_norm_rope(qkv[:0], 4, 2, cu, inv_freq=torch.zeros(32), positions=pos[:, :0], pair_axis=axis)
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128)
