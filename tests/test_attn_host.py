"""Host-side checks of the softmax-attention entry points: every bad argument is
refused with the documented status before any HIP call, and the binding refuses
tensors that do not fit. No test here launches a kernel."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import chunked_gated_delta_rule_amd as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = 0, 1, 2, 3, 4
P = 0x10000  # a pointer that the host checks accept and never follow


def cfg(**kw):
    c = gdn.make_attn_config(64, 4, 8, 2, 128, gdn.GDN_BF16, rot_dim=64, page_size=16, n_pages=9,
                             max_pages=3)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def refused(status, fn, *a, **kw):
    with pytest.raises(gdn.GDNError) as e:
        fn(*a, stream=0, **kw)
    assert e.value.status == status


@pytest.mark.parametrize("field,value,status", [
    ("t_max", -1, INVALID), ("n_max", 0, INVALID), ("h", 0, INVALID), ("hkv", 0, INVALID),
    ("dtype", 9, INVALID), ("dtype", gdn.GDN_F32, UNSUPPORTED), ("dtype", gdn.GDN_F16, OK),
    ("d", 64, UNSUPPORTED), ("d", 256, OK), ("h", 9, UNSUPPORTED), ("h", 2, OK),
    ("scale", float("nan"), INVALID), ("scale", float("inf"), INVALID),
    ("eps", -1e-6, INVALID), ("eps", float("inf"), INVALID), ("eps", 0.0, OK),
    ("rot_dim", -2, INVALID), ("rot_dim", 63, INVALID), ("rot_dim", 130, INVALID),
    ("rot_dim", 128, OK), ("rot_dim", 2, OK), ("rot_interleaved", 2, INVALID),
    ("rot_scale", float("nan"), INVALID),
    ("page_size", 0, UNSUPPORTED), ("page_size", 8, UNSUPPORTED), ("page_size", 48, UNSUPPORTED),
    ("page_size", 512, UNSUPPORTED), ("page_size", 256, OK),
    ("n_pages", -1, INVALID), ("max_pages", -1, INVALID), ("tk_max", -1, INVALID),
    ("shared_max", -1, INVALID),
    ("t_max", (1 << 24) + 1, CAPACITY), ("tk_max", (1 << 24) + 1, CAPACITY),
    ("n_max", 16385, CAPACITY), ("h", 4098, CAPACITY), ("max_pages", (1 << 26) + 1, CAPACITY),
])
def test_config_validation(field, value, status):
    c = cfg(**{field: value})
    out = ctypes.c_size_t(0)
    assert gdn.load_library().gdn_attn_workspace_size(ctypes.byref(c), ctypes.byref(out)) == status


def test_rows_times_heads_are_counted_in_32_bits():
    refused_cfg = cfg(t_max=1 << 24, h=128)
    out = ctypes.c_size_t(0)
    lib = gdn.load_library()
    assert lib.gdn_attn_workspace_size(ctypes.byref(refused_cfg), ctypes.byref(out)) == CAPACITY
    assert lib.gdn_attn_workspace_size(None, ctypes.byref(out)) == INVALID
    assert lib.gdn_attn_workspace_size(ctypes.byref(cfg()), None) == INVALID


def test_workspace_depends_on_the_prefix_capacity():
    c = dict(max_pages=1 << 14)
    a = gdn.gdn_attn_workspace_size(cfg(**c))
    assert a > 0 and a % 256 == 0
    # a prefix of at most 100 positions is not worth a pass of its own
    assert gdn.gdn_attn_workspace_size(cfg(shared_max=100, **c)) == a
    rows = 64 * 8 * 2
    assert gdn.gdn_attn_workspace_size(cfg(shared_max=1 << 18, **c)) - a >= rows * 128 * 4


FRONT = dict(qkv=P, q_w=P, k_w=P, inv_freq=P, cu_seqlens=P, kv_lens=P, q=P, k=P)


@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(cu_seqlens=None), dict(q=None), dict(k=None), dict(inv_freq=None),
    dict(qkv=P + 8), dict(q=P + 2), dict(k=P + 4), dict(q_w=P + 1), dict(k_w=P + 2),
    dict(inv_freq=P + 3), dict(cu_seqlens=P + 2), dict(kv_lens=P + 1),
])
def test_norm_rope_refusals(change):
    refused(INVALID, gdn.gdn_qk_norm_rope, cfg(), **{**FRONT, **change})


def test_norm_rope_needs_frequencies_exactly_when_it_rotates():
    refused(INVALID, gdn.gdn_qk_norm_rope, cfg(rot_dim=0), **FRONT)


@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(cu_seqlens=None), dict(kv_lens=None), dict(block_table=None),
    dict(k_pages=None), dict(v_pages=None), dict(k_pages=P + 8), dict(v_pages=P + 2),
    dict(block_table=P + 2), dict(q=P + 8), dict(k=P + 8),
])
def test_append_refusals(change):
    a = {**FRONT, "block_table": P, "k_pages": P, "v_pages": P, **change}
    refused(INVALID, gdn.gdn_kv_append, cfg(), **a)


@pytest.mark.parametrize("field", ["n_pages", "max_pages"])
def test_cache_calls_need_pages(field):
    a = {**FRONT, "block_table": P, "k_pages": P, "v_pages": P}
    refused(INVALID, gdn.gdn_kv_append, cfg(**{field: 0}), **a)
    refused(INVALID, gdn.gdn_attn_paged, cfg(**{field: 0}), P, P, P, P, P, P, None, P, P, 1 << 40)


PREFILL = dict(q=P, k=P, v=P, cu_q=P, cu_k=None, o=P, workspace=P, ws_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(cu_q=None), INVALID), (dict(o=None), INVALID), (dict(q=P + 8), INVALID),
    (dict(k=P + 2), INVALID), (dict(v=P + 4), INVALID), (dict(o=P + 8), INVALID),
    (dict(cu_q=P + 1), INVALID), (dict(cu_k=P + 2), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=P + 128), WORKSPACE),
    (dict(ws_bytes=100), WORKSPACE),
])
def test_prefill_refusals(change, status):
    refused(status, gdn.gdn_attn_prefill, cfg(), **{**PREFILL, **change})


PAGED = dict(q=P, k_pages=P, v_pages=P, cu_seqlens=P, kv_lens=P, block_table=P, shared_len=None,
             o=P, workspace=P, ws_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID),
    (dict(cu_seqlens=None), INVALID), (dict(kv_lens=None), INVALID),
    (dict(block_table=None), INVALID), (dict(o=None), INVALID), (dict(q=P + 8), INVALID),
    (dict(k_pages=P + 8), INVALID), (dict(v_pages=P + 8), INVALID), (dict(o=P + 2), INVALID),
    (dict(shared_len=P + 2), INVALID), (dict(kv_lens=P + 2), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=P + 64), WORKSPACE),
    (dict(ws_bytes=255), WORKSPACE),
])
def test_paged_refusals(change, status):
    refused(status, gdn.gdn_attn_paged, cfg(), **{**PAGED, **change})


@pytest.mark.parametrize("row,status", [(8 * 128 - 8, INVALID), (8 * 128 + 4, INVALID),
                                        (-8, INVALID)])
def test_row_strides_are_checked(row, status):
    lib, c = gdn.load_library(), cfg()
    b = ctypes.byref(c)
    assert lib.gdn_attn_prefill(b, P, row, P, 0, P, 0, P, None, P, P, 1 << 40, None) == status
    assert lib.gdn_attn_paged(b, P, row, P, P, P, P, P, None, P, P, 1 << 40, None) == status
    assert lib.gdn_qk_norm_rope(b, P, row, P, P, P, P, P, P, P, None) == status


def test_nothing_to_do_is_fine_without_a_device():
    c = cfg(t_max=0)
    gdn.gdn_qk_norm_rope(c, **FRONT, stream=0)
    gdn.gdn_kv_append(c, **FRONT, block_table=P, k_pages=P, v_pages=P, stream=0)
    gdn.gdn_attn_prefill(c, **PREFILL, stream=0)
    gdn.gdn_attn_paged(c, **PAGED, stream=0)


def test_binding_refuses_tensors_that_do_not_fit():
    """Host tensors stand in: every check but the last one (device) comes first."""
    c = cfg()
    t = torch.bfloat16
    good = dict(q=torch.zeros(64, 8, 128, dtype=t), k=torch.zeros(64, 2, 128, dtype=t),
                v=torch.zeros(64, 2, 128, dtype=t), cu_q=torch.zeros(5, dtype=torch.int32),
                cu_k=None, o=torch.zeros(64, 8, 128, dtype=t), workspace=P, ws_bytes=1 << 40)

    def bad(match, **change):
        with pytest.raises(ValueError, match=match):
            gdn.gdn_attn_prefill(c, **{**good, **change}, stream=0)

    bad("device tensor")
    bad("dtype", q=good["q"].half())
    bad("expected", q=good["q"][:63])
    bad("expected", q=good["q"].transpose(0, 1))
    bad("expected", k=good["q"])
    bad("expected", k=torch.zeros(64, 2, 256, dtype=t)[..., ::2])
    bad("expected", v=torch.zeros(1, 2, 128, dtype=t).expand(64, 2, 128))
    with pytest.raises(ValueError, match="dtype"):
        gdn.make_attn_config(1, 1, 1, 1, dtype=torch.float32)
    with pytest.raises(ValueError, match="one dtype"):
        gdn.causal_attention(good["q"], good["k"], good["v"].half(), good["cu_q"])
    with pytest.raises(ValueError, match="rows"):
        gdn.causal_attention(good["q"], good["k"][:9], good["v"][:9], good["cu_q"])
    with pytest.raises(ValueError, match="number of sequences"):
        gdn.causal_attention(good["q"], good["k"], good["v"], good["cu_q"], good["cu_q"][:3])
    with pytest.raises(ValueError, match="qkv"):
        gdn.qk_norm_rope(torch.zeros(4, 100, dtype=t), 8, 2, good["cu_q"])
    pages = torch.zeros(3, 2, 16, 128, dtype=t)
    table = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="pages"):
        gdn.paged_attention(good["q"], pages, pages[:, :, :8], good["cu_q"], table[:, 0], table)
    with pytest.raises(ValueError, match="head dim|d\\]"):
        gdn.append_paged_kv(torch.zeros(4, 10 * 256, dtype=t), 6, good["cu_q"], table[:, 0], table,
                            pages, pages)


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), 1e-60])
def test_high_level_calls_refuse_a_scale_that_is_not_positive(scale):
    t = torch.bfloat16
    q, cu = torch.zeros(4, 2, 128, dtype=t), torch.zeros(2, dtype=torch.int32)
    pages, table = torch.zeros(3, 2, 16, 128, dtype=t), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="scale"):
        gdn.causal_attention(q, q, q, cu, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        gdn.paged_attention(q, pages, pages, cu, cu[:1], table, scale=scale)


def test_high_level_calls_of_no_tokens_give_empty_results():
    t = torch.float16
    cu = torch.zeros(3, dtype=torch.int32)
    pages, table = torch.zeros(3, 2, 16, 128, dtype=t), torch.zeros(2, 2, dtype=torch.int32)
    qkv, q = torch.zeros(0, 8 * 128, dtype=t), torch.zeros(0, 4, 128, dtype=t)
    a, b = gdn.qk_norm_rope(qkv, 4, 2, cu)
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128) and a.dtype == t
    a, b = gdn.append_paged_kv(qkv, 4, cu, cu[:2], table, pages, pages.clone(), output_k=True)
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128)
    assert gdn.causal_attention(q, q[:, :2], q[:, :2], cu).shape == (0, 4, 128)
    assert gdn.paged_attention(q, pages, pages, cu, cu[:2], table).shape == (0, 4, 128)


def test_binding_struct_matches_the_header(tmp_path):
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    text = open(os.path.join(ROOT, "include", "gdn.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} gdn_attn_config;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip() for line in re.findall(r"\w+ ([^;]+);", body) for n in line.split(",")]
    assert names == [n for n, _ in gdn.gdn_attn_config._fields_]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gdn.h"', "int main(void) {",
             '  printf("size %zu\\n", sizeof(gdn_attn_config));']
    lines += [f'  printf("{n} %zu\\n", offsetof(gdn_attn_config, {n}));' for n in names]
    src, exe = tmp_path / "a.c", tmp_path / "a"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], check=True, capture_output=True,
                                                 text=True).stdout.splitlines())
    assert int(got.pop("size")) == ctypes.sizeof(gdn.gdn_attn_config)
    for n in names:
        assert int(got[n]) == getattr(gdn.gdn_attn_config, n).offset, n


@pytest.mark.parametrize("scale,status", [(3e38, INVALID), (2.4e38, INVALID), (2.3e38, OK), (1e-44, OK)])
def test_a_scale_that_leaves_fp32_with_the_exponents_base_is_refused(scale, status):
    """Kernels take scale * log2(e) in fp32: finite up to 2^128 / log2(e) = 2.3586e38."""
    out = ctypes.c_size_t(0)
    lib = gdn.load_library()
    assert lib.gdn_attn_workspace_size(ctypes.byref(cfg(scale=scale)), ctypes.byref(out)) == status
    if status != OK:
        refused(status, gdn.gdn_attn_prefill, cfg(scale=scale), **PREFILL)
        refused(status, gdn.gdn_attn_paged, cfg(scale=scale), **PAGED)
