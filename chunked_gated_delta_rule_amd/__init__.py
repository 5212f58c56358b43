"""Python binding of libgdn.so, the MI355X (gfx950) chunked gated-delta-rule
prefill forward.

The functions below carry the names of the C ABI in ``include/gdn.h`` and
only marshal arguments: torch tensors become device pointers, the current
torch stream becomes the hipStream_t, and a non-OK status becomes a
``GDNError``. Every step of the computation runs in the library's HIP
kernels; there is no fallback of any kind. If the library has not been built
(``python -m chunked_gated_delta_rule_amd.build``), importing the binding
still works but the first call raises.

Layouts (packed varlen, batch 1): q, k [t_max, h, 128]; v, o [t_max, hv, 128];
g, beta [t_max, hv] fp32; states [n_max, hv, 128 (v), 128 (k)] fp32;
cu_seqlens int32 [n_max + 1].
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

__all__ = [
    "GDNError", "gdn_config", "GDN_BF16", "GDN_F32", "GDN_F16", "load_library", "library_path",
    "gdn_nt_max", "gdn_workspace_size", "gdn_build_chunk_indices", "gdn_front_conv_silu_l2",
    "gdn_chunk_fwd_intra", "gdn_chunk_fwd_inter", "gdn_chunk_fwd", "gdn_status_str",
    "gdn_workspace_layout", "make_config", "chunk_gated_delta_rule", "EXPORTED_SYMBOLS",
    "gdn_chunk_fwd_timed", "gdn_front_conv_silu_l2_timed", "GDN_FUSED_INDEX_MAX_SEQS",
    "gdn_chunk_fwd_conv", "gdn_chunk_fwd_conv_timed", "gdn_recurrent_fwd",
    "gdn_recurrent_fwd_timed", "recurrent_gated_delta_rule", "GDN_SEGMENT_MIN_TOKENS", "GDN_FOUR_TILE_MIN_TOKENS",
    "GDN_T_MAX_LIMIT", "GDN_N_MAX_LIMIT", "gdn_chunk_fwd_noalloc", "GDN_NOALLOC_SCRATCH_BYTES",
    "gdn_attn_config", "make_attn_config", "gdn_attn_workspace_size", "gdn_qk_norm_rope",
    "gdn_kv_append", "gdn_attn_prefill", "gdn_attn_paged", "rope_inv_freq", "qk_norm_rope",
    "append_paged_kv", "causal_attention", "paged_attention",
]

GDN_BF16 = 0
GDN_F32 = 1
GDN_F16 = 2
GDN_FUSED_INDEX_MAX_SEQS = 256  # include/gdn.h
GDN_SEGMENT_MIN_TOKENS = 2048  # include/gdn.h
GDN_FOUR_TILE_MIN_TOKENS = 384  # include/gdn.h
GDN_T_MAX_LIMIT = 1 << 24  # include/gdn.h
GDN_N_MAX_LIMIT = 16384  # include/gdn.h
GDN_NOALLOC_SCRATCH_BYTES = 256 << 20  # include/gdn.h
_STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED",
           3: "GDN_ERR_CAPACITY", 4: "GDN_ERR_WORKSPACE", 5: "GDN_ERR_HIP"}
EXPORTED_SYMBOLS = ("gdn_nt_max", "gdn_workspace_layout", "gdn_workspace_size",
                    "gdn_build_chunk_indices", "gdn_front_conv_silu_l2", "gdn_chunk_fwd_intra",
                    "gdn_chunk_fwd_inter", "gdn_chunk_fwd", "gdn_status_str",
                    "gdn_chunk_fwd_timed", "gdn_front_conv_silu_l2_timed", "gdn_chunk_fwd_conv",
                    "gdn_chunk_fwd_conv_timed", "gdn_recurrent_fwd", "gdn_recurrent_fwd_timed",
                    "gdn_chunk_fwd_noalloc", "gdn_attn_workspace_size", "gdn_qk_norm_rope",
                    "gdn_kv_append", "gdn_attn_prefill", "gdn_attn_paged")

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libgdn.so")


class gdn_config(ctypes.Structure):
    _fields_ = [("t_max", ctypes.c_int32), ("n_max", ctypes.c_int32), ("h", ctypes.c_int32),
                ("hv", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("qkv_dtype", ctypes.c_int), ("o_dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("segments", ctypes.c_int32),
                ("tiles", ctypes.c_int32), ("gqa_share", ctypes.c_int32)]


class gdn_workspace_layout_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("w16", "q16", "kimg", "uimg", "pimg", "gimg", "table", "order", "seg_sa", "seg_z",
                 "seg_phi", "seg_oh", "total")]


class gdn_attn_config(ctypes.Structure):
    _fields_ = [("t_max", ctypes.c_int32), ("n_max", ctypes.c_int32), ("h", ctypes.c_int32),
                ("hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("rot_dim", ctypes.c_int32),
                ("rot_interleaved", ctypes.c_int32), ("rot_scale", ctypes.c_float),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("tk_max", ctypes.c_int32),
                ("shared_max", ctypes.c_int32)]


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}")


_lib = None


def load_library():
    """Load libgdn.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is missing: build it with "
                           "`python -m chunked_gated_delta_rule_amd.build`")
    lib = ctypes.CDLL(library_path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    cfgp = ctypes.POINTER(gdn_config)
    lib.gdn_nt_max.argtypes = [i32, i32, i32]
    lib.gdn_nt_max.restype = ctypes.c_int64
    lib.gdn_workspace_size.argtypes = [cfgp, ctypes.POINTER(sz)]
    lib.gdn_workspace_layout.argtypes = [cfgp, ctypes.POINTER(gdn_workspace_layout_t)]
    lib.gdn_build_chunk_indices.argtypes = [cfgp, vp, vp, vp]
    lib.gdn_front_conv_silu_l2.argtypes = [cfgp, vp, vp, i32, vp, vp, vp, vp, vp]
    lib.gdn_chunk_fwd_intra.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdn_chunk_fwd_inter.argtypes = [cfgp, vp, vp, vp, sz, vp, vp, vp]
    lib.gdn_chunk_fwd.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdn_chunk_fwd_timed.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                        ctypes.POINTER(vp)]
    lib.gdn_front_conv_silu_l2_timed.argtypes = [cfgp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.gdn_chunk_fwd_conv.argtypes = [cfgp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdn_chunk_fwd_conv_timed.argtypes = [cfgp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                             vp, ctypes.POINTER(vp)]
    lib.gdn_recurrent_fwd.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.gdn_chunk_fwd_noalloc.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.gdn_recurrent_fwd_timed.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    acfg, i64 = ctypes.POINTER(gdn_attn_config), ctypes.c_int64
    lib.gdn_attn_workspace_size.argtypes = [acfg, ctypes.POINTER(sz)]
    lib.gdn_qk_norm_rope.argtypes = [acfg, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.gdn_kv_append.argtypes = [acfg, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.gdn_attn_prefill.argtypes = [acfg, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, sz, vp]
    lib.gdn_attn_paged.argtypes = [acfg, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for name in ("gdn_attn_workspace_size", "gdn_qk_norm_rope", "gdn_kv_append",
                 "gdn_attn_prefill", "gdn_attn_paged"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("gdn_workspace_size", "gdn_workspace_layout", "gdn_build_chunk_indices", "gdn_front_conv_silu_l2",
                 "gdn_chunk_fwd_intra", "gdn_chunk_fwd_inter", "gdn_chunk_fwd",
                 "gdn_chunk_fwd_timed", "gdn_front_conv_silu_l2_timed", "gdn_chunk_fwd_conv",
                 "gdn_chunk_fwd_conv_timed", "gdn_recurrent_fwd", "gdn_recurrent_fwd_timed",
                 "gdn_chunk_fwd_noalloc"):
        getattr(lib, name).restype = ctypes.c_int
    lib.gdn_status_str.argtypes = [ctypes.c_int]
    lib.gdn_status_str.restype = ctypes.c_char_p
    _lib = lib
    return lib


_TORCH_DTYPE = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32, torch.float16: GDN_F16}
_GDN_DTYPE = {GDN_BF16: torch.bfloat16, GDN_F32: torch.float32, GDN_F16: torch.float16}


def make_config(t_max, n_max, h, hv, qkv_dtype=GDN_BF16, scale=0.0, o_dtype=GDN_F32,
                dk=128, dv=128, chunk=64, segments=0, tiles=0, gqa_share=0) -> gdn_config:
    """A gdn_config; qkv_dtype is GDN_BF16 / GDN_F32 / GDN_F16 or the torch
    dtype (bfloat16, float32, float16; any other raises ValueError)."""
    if isinstance(qkv_dtype, torch.dtype):
        if qkv_dtype not in _TORCH_DTYPE:
            raise ValueError(f"q/k/v dtype {qkv_dtype}: bfloat16, float32 or float16 expected")
        qkv_dtype = _TORCH_DTYPE[qkv_dtype]
    return gdn_config(int(t_max), int(n_max), int(h), int(hv), int(dk), int(dv), int(chunk),
                      int(qkv_dtype), int(o_dtype), float(scale), int(segments), int(tiles),
                      int(gqa_share))


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, torch.Tensor):
        if not x.is_cuda:
            raise ValueError("device tensor expected")
        if not x.is_contiguous():
            raise ValueError("contiguous tensor expected")
        return x.data_ptr()
    raise TypeError(type(x))


def _need(x, name, elems, dtype, last=None):
    """A tensor argument must have `dtype`, hold at least `elems` elements (the
    kernels index that many from its start) and, when `last` is given and the
    tensor has more than one dimension, end in a dimension of that size. Raw
    pointers (ints) and None are passed through unchecked."""
    if not isinstance(x, torch.Tensor):
        return
    if x.dtype != dtype:
        raise ValueError(f"{name}: dtype {x.dtype}, {dtype} expected")
    if x.numel() < elems:
        raise ValueError(f"{name}: {x.numel()} elements, at least {elems} expected")
    if last is not None and x.dim() > 1 and x.shape[-1] != last:
        raise ValueError(f"{name}: last dimension {x.shape[-1]}, {last} expected")


def _check_tensors(cfg, q=None, k=None, v=None, g=None, beta=None, h0=None, cu=None,
                   table=None, o=None, hT=None):
    """Dtypes and sizes of the tensor arguments against `cfg` (include/gdn.h layouts)."""
    T, n, h, hv, dk, dv = cfg.t_max, cfg.n_max, cfg.h, cfg.hv, cfg.dk, cfg.dv
    qdt = _GDN_DTYPE.get(cfg.qkv_dtype, torch.bfloat16)
    _need(q, "q", T * h * dk, qdt, dk)
    _need(k, "k", T * h * dk, qdt, dk)
    _need(v, "v", T * hv * dv, qdt, dv)
    _need(g, "g", T * hv, torch.float32)
    _need(beta, "beta", T * hv, torch.float32)
    _need(h0, "h0", n * hv * dv * dk, torch.float32, dk)
    _need(hT, "hT", n * hv * dv * dk, torch.float32, dk)
    _need(cu, "cu_seqlens", n + 1, torch.int32)
    if table is not None:
        _need(table, "chunk_indices", 2 * max(gdn_nt_max(T, n, cfg.chunk), 0), torch.int32)
    _need(o, "o", T * hv * dv, torch.float32, dv)


def _check_front(cfg, qkv, conv_w, d_conv):
    C = (2 * cfg.h * cfg.dk + cfg.hv * cfg.dv)
    _need(qkv, "qkv", cfg.t_max * C, torch.bfloat16, C)
    _need(conv_w, "conv_w", C * int(d_conv), torch.bfloat16)


def _check_ws(workspace, ws_bytes):
    if isinstance(workspace, torch.Tensor) and \
            workspace.numel() * workspace.element_size() < int(ws_bytes):
        raise ValueError(f"workspace: {workspace.numel() * workspace.element_size()} bytes, "
                         f"ws_bytes = {int(ws_bytes)}")


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, where: str):
    if st != 0:
        raise GDNError(st, where)


def gdn_status_str(status: int) -> str:
    return load_library().gdn_status_str(int(status)).decode()


def gdn_nt_max(t_max: int, n_max: int, chunk: int = 64) -> int:
    return int(load_library().gdn_nt_max(int(t_max), int(n_max), int(chunk)))


def gdn_workspace_size(cfg: gdn_config) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gdn_workspace_size(ctypes.byref(cfg), ctypes.byref(out)),
           "gdn_workspace_size")
    return int(out.value)


def gdn_build_chunk_indices(cfg, cu_seqlens, chunk_indices, stream=None):
    _check_tensors(cfg, cu=cu_seqlens, table=chunk_indices)
    _check(load_library().gdn_build_chunk_indices(ctypes.byref(cfg), _ptr(cu_seqlens),
                                                  _ptr(chunk_indices), _stream(stream)),
           "gdn_build_chunk_indices")


def gdn_front_conv_silu_l2(cfg, qkv, conv_w, d_conv, cu_seqlens, q, k, v, stream=None):
    _check_front(cfg, qkv, conv_w, d_conv)
    _check_tensors(make_config(cfg.t_max, cfg.n_max, cfg.h, cfg.hv, GDN_F32), q=q, k=k, v=v,
                   cu=cu_seqlens)
    _check(load_library().gdn_front_conv_silu_l2(ctypes.byref(cfg), _ptr(qkv), _ptr(conv_w),
                                                 int(d_conv), _ptr(cu_seqlens), _ptr(q), _ptr(k),
                                                 _ptr(v), _stream(stream)),
           "gdn_front_conv_silu_l2")


def gdn_workspace_layout(cfg: gdn_config) -> dict:
    """Byte offsets of the intermediates inside a workspace (and its total size)."""
    out = gdn_workspace_layout_t()
    _check(load_library().gdn_workspace_layout(ctypes.byref(cfg), ctypes.byref(out)),
           "gdn_workspace_layout")
    return {name: int(getattr(out, name)) for name, _ in gdn_workspace_layout_t._fields_}


def _ws_bytes(workspace, ws_bytes):
    if ws_bytes is not None:
        return int(ws_bytes)
    return workspace.numel() * workspace.element_size()


def gdn_chunk_fwd_intra(cfg, q, k, v, g, beta, cu_seqlens, chunk_indices, workspace,
                        ws_bytes=None, stream=None):
    _check_tensors(cfg, q=q, k=k, v=v, g=g, beta=beta, cu=cu_seqlens, table=chunk_indices)
    _check_ws(workspace, _ws_bytes(workspace, ws_bytes))
    _check(load_library().gdn_chunk_fwd_intra(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                              _ptr(chunk_indices), _ptr(workspace),
                                              _ws_bytes(workspace, ws_bytes), _stream(stream)),
           "gdn_chunk_fwd_intra")


def gdn_chunk_fwd_inter(cfg, h0, cu_seqlens, workspace, o, hT, ws_bytes=None, stream=None):
    _check_tensors(cfg, h0=h0, cu=cu_seqlens, o=o, hT=hT)
    _check_ws(workspace, _ws_bytes(workspace, ws_bytes))
    _check(load_library().gdn_chunk_fwd_inter(ctypes.byref(cfg), _ptr(h0), _ptr(cu_seqlens),
                                              _ptr(workspace), _ws_bytes(workspace, ws_bytes),
                                              _ptr(o), _ptr(hT), _stream(stream)),
           "gdn_chunk_fwd_inter")


def gdn_chunk_fwd(cfg, q, k, v, g, beta, h0, cu_seqlens, chunk_indices, o, hT, workspace,
                  ws_bytes=None, stream=None):
    ws_bytes = _ws_bytes(workspace, ws_bytes)
    _check_tensors(cfg, q, k, v, g, beta, h0, cu_seqlens, chunk_indices, o, hT)
    _check_ws(workspace, ws_bytes)
    _check(load_library().gdn_chunk_fwd(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                        _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
                                        _ptr(chunk_indices), _ptr(o), _ptr(hT), _ptr(workspace),
                                        int(ws_bytes), _stream(stream)),
           "gdn_chunk_fwd")


def gdn_chunk_fwd_noalloc(cfg, q, k, v, g, beta, h0, cu_seqlens, chunk_indices, o, hT,
                          stream=None):
    """gdn_chunk_fwd with the intermediates in the library's fixed device
    scratch (no workspace argument; nothing is allocated)."""
    _check_tensors(cfg, q, k, v, g, beta, h0, cu_seqlens, chunk_indices, o, hT)
    _check(load_library().gdn_chunk_fwd_noalloc(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v),
                                                _ptr(g), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
                                                _ptr(chunk_indices), _ptr(o), _ptr(hT),
                                                _stream(stream)),
           "gdn_chunk_fwd_noalloc")


def gdn_chunk_fwd_timed(cfg, q, k, v, g, beta, h0, cu_seqlens, chunk_indices, o, hT, workspace,
                        events, ws_bytes=None, stream=None):
    """gdn_chunk_fwd whose kernels record `events` (six raw hipEvent_t handles,
    ints) at their own start and end: table, intra, inter."""
    ws_bytes = _ws_bytes(workspace, ws_bytes)
    _check_tensors(cfg, q, k, v, g, beta, h0, cu_seqlens, chunk_indices, o, hT)
    _check_ws(workspace, ws_bytes)
    if len(events) != 6:
        raise ValueError("six events expected")
    arr = (ctypes.c_void_p * 6)(*[int(e) for e in events])
    _check(load_library().gdn_chunk_fwd_timed(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(g), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
                                              _ptr(chunk_indices), _ptr(o), _ptr(hT),
                                              _ptr(workspace), int(ws_bytes), _stream(stream),
                                              arr),
           "gdn_chunk_fwd_timed")


def gdn_front_conv_silu_l2_timed(cfg, qkv, conv_w, d_conv, cu_seqlens, q, k, v, ev_start, ev_stop,
                                 stream=None):
    _check_front(cfg, qkv, conv_w, d_conv)
    _check_tensors(make_config(cfg.t_max, cfg.n_max, cfg.h, cfg.hv, GDN_F32), q=q, k=k, v=v,
                   cu=cu_seqlens)
    _check(load_library().gdn_front_conv_silu_l2_timed(
        ctypes.byref(cfg), _ptr(qkv), _ptr(conv_w), int(d_conv), _ptr(cu_seqlens), _ptr(q),
        _ptr(k), _ptr(v), _stream(stream), int(ev_start), int(ev_stop)),
        "gdn_front_conv_silu_l2_timed")


def gdn_chunk_fwd_conv(cfg, qkv, conv_w, d_conv, g, beta, h0, cu_seqlens, chunk_indices, o, hT,
                       workspace, ws_bytes=None, stream=None):
    ws_bytes = _ws_bytes(workspace, ws_bytes)
    _check_front(cfg, qkv, conv_w, d_conv)
    _check_tensors(cfg, g=g, beta=beta, h0=h0, cu=cu_seqlens, table=chunk_indices, o=o, hT=hT)
    _check_ws(workspace, ws_bytes)
    _check(load_library().gdn_chunk_fwd_conv(ctypes.byref(cfg), _ptr(qkv), _ptr(conv_w),
                                             int(d_conv), _ptr(g), _ptr(beta), _ptr(h0),
                                             _ptr(cu_seqlens), _ptr(chunk_indices), _ptr(o),
                                             _ptr(hT), _ptr(workspace), int(ws_bytes),
                                             _stream(stream)),
           "gdn_chunk_fwd_conv")


def gdn_chunk_fwd_conv_timed(cfg, qkv, conv_w, d_conv, g, beta, h0, cu_seqlens, chunk_indices, o,
                             hT, workspace, events, ws_bytes=None, stream=None):
    """gdn_chunk_fwd_conv whose kernels record `events` (six raw hipEvent_t
    handles): table, intra (with the fused front), inter."""
    ws_bytes = _ws_bytes(workspace, ws_bytes)
    _check_front(cfg, qkv, conv_w, d_conv)
    _check_tensors(cfg, g=g, beta=beta, h0=h0, cu=cu_seqlens, table=chunk_indices, o=o, hT=hT)
    _check_ws(workspace, ws_bytes)
    if len(events) != 6:
        raise ValueError("six events expected")
    arr = (ctypes.c_void_p * 6)(*[int(e) for e in events])
    _check(load_library().gdn_chunk_fwd_conv_timed(ctypes.byref(cfg), _ptr(qkv), _ptr(conv_w),
                                                   int(d_conv), _ptr(g), _ptr(beta), _ptr(h0),
                                                   _ptr(cu_seqlens), _ptr(chunk_indices), _ptr(o),
                                                   _ptr(hT), _ptr(workspace), int(ws_bytes),
                                                   _stream(stream), arr),
           "gdn_chunk_fwd_conv_timed")


def gdn_recurrent_fwd(cfg, q, k, v, g, beta, h0, cu_seqlens, o, hT, stream=None):
    _check_tensors(cfg, q, k, v, g, beta, h0, cu_seqlens, None, o, hT)
    _check(load_library().gdn_recurrent_fwd(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                            _ptr(beta), _ptr(h0), _ptr(cu_seqlens), _ptr(o),
                                            _ptr(hT), _stream(stream)),
           "gdn_recurrent_fwd")


def gdn_recurrent_fwd_timed(cfg, q, k, v, g, beta, h0, cu_seqlens, o, hT, ev_start, ev_stop,
                            stream=None):
    """gdn_recurrent_fwd whose kernel records raw hipEvent_t handles at its start and end."""
    _check_tensors(cfg, q, k, v, g, beta, h0, cu_seqlens, None, o, hT)
    _check(load_library().gdn_recurrent_fwd_timed(
        ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
        _ptr(cu_seqlens), _ptr(o), _ptr(hT), _stream(stream), int(ev_start), int(ev_stop)),
        "gdn_recurrent_fwd_timed")


def _same_qkv_dtype(q, k, v):
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in _TORCH_DTYPE:
        raise ValueError(f"q, k, v must share one dtype in (bfloat16, float32, float16): "
                         f"{q.dtype}, {k.dtype}, {v.dtype}")
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[0] != q.shape[0]:
        raise ValueError(f"q, k [T, H, 128] and v [T, Hv, 128] expected: {tuple(q.shape)}, "
                         f"{tuple(k.shape)}, {tuple(v.shape)}")


def recurrent_gated_delta_rule(q, k, v, g, beta, cu_seqlens, initial_state=None,
                               output_final_state=True, scale=None, n_max=None):
    """Allocate outputs with torch and run gdn_recurrent_fwd (token-serial decode /
    verify) on the current stream. Arguments as chunk_gated_delta_rule, with
    q, k, v in bf16 or fp32 (the token-serial kernel takes no fp16)."""
    _same_qkv_dtype(q, k, v)
    T, H, _ = q.shape
    Hv = v.shape[1]
    n = cu_seqlens.numel() - 1 if n_max is None else n_max
    cfg = make_config(T, n, H, Hv, q.dtype, scale or 0.0)
    o = torch.empty((T, Hv, 128), dtype=torch.float32, device=q.device)
    hT = torch.empty((n, Hv, 128, 128), dtype=torch.float32, device=q.device) \
        if output_final_state else None
    gdn_recurrent_fwd(cfg, q, k, v, g, beta, initial_state, cu_seqlens, o, hT)
    return o, hT


def chunk_gated_delta_rule(q, k, v, g, beta, cu_seqlens, initial_state=None,
                           output_final_state=True, scale=None, chunk_indices=None,
                           workspace=None, n_max=None):
    """Allocate outputs with torch and run gdn_chunk_fwd on the current stream.

    q, k [T, H, 128] and v [T, Hv, 128] (bf16, fp16 or fp32, one dtype); g, beta
    [T, Hv] fp32; cu_seqlens int32 [N + 1] on the device; initial_state
    [N, Hv, 128, 128] fp32 or None. Returns (o [T, Hv, 128] fp32, final state
    or None).
    """
    _same_qkv_dtype(q, k, v)
    T, H, _ = q.shape
    Hv = v.shape[1]
    n = cu_seqlens.numel() - 1 if n_max is None else n_max
    cfg = make_config(T, n, H, Hv, q.dtype, scale or 0.0)
    if workspace is None:
        workspace = torch.empty(gdn_workspace_size(cfg), dtype=torch.uint8, device=q.device)
    o = torch.empty((T, Hv, 128), dtype=torch.float32, device=q.device)
    hT = torch.empty((n, Hv, 128, 128), dtype=torch.float32, device=q.device) \
        if output_final_state else None
    gdn_chunk_fwd(cfg, q, k, v, g, beta, initial_state, cu_seqlens, chunk_indices, o, hT,
                  workspace)
    return o, hT


# ---- softmax-attention layers of a hybrid stack (include/gdn.h, last section). Forward
# only, like the calls above: results carry no gradient.

def make_attn_config(t_max, n_max, h, hkv, d=128, dtype=GDN_BF16, scale=0.0, eps=1e-6, rot_dim=0,
                     rot_interleaved=False, rot_scale=0.0, page_size=16, n_pages=0, max_pages=0,
                     tk_max=0, shared_max=0) -> gdn_attn_config:
    """A gdn_attn_config; dtype is GDN_BF16 / GDN_F16 or the torch dtype."""
    if isinstance(dtype, torch.dtype):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"attention dtype {dtype}: bfloat16 or float16 expected")
        dtype = _TORCH_DTYPE[dtype]
    return gdn_attn_config(int(t_max), int(n_max), int(h), int(hkv), int(d), int(dtype),
                           float(scale), float(eps), int(rot_dim), int(bool(rot_interleaved)),
                           float(rot_scale), int(page_size), int(n_pages), int(max_pages),
                           int(tk_max), int(shared_max))


def gdn_attn_workspace_size(cfg: gdn_attn_config) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gdn_attn_workspace_size(ctypes.byref(cfg), ctypes.byref(out)),
           "gdn_attn_workspace_size")
    return int(out.value)


# A small attention call is bound by the host, so its argument checks are kept to
# one short function per tensor, with the message put together only on failure.

# torch's raw handle of the current stream of a device, and its current device (the
# Stream object for the former costs as much as a kernel launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _dev(*tensors):
    """Index of the device of the first tensor (None: raw pointers only; below 0: a
    host tensor, which the call refuses after the other checks)."""
    for x in tensors:
        if x.__class__ is not int and x is not None:
            return x.get_device()
    return None


def _at(x, name, dtype, elems, dev, last=None):
    """Pointer of a contiguous tensor on device `dev` with at least `elems` elements
    of `dtype` (None and raw pointers pass through)."""
    if x is None or x.__class__ is int:
        return x
    if x.dtype is dtype and x.get_device() == dev and x.is_contiguous() and \
            x.numel() >= elems and (last is None or x.size(-1) == last):
        return x.data_ptr()
    _need(x, name, elems, dtype, last)
    if x.get_device() != dev:
        raise ValueError(f"{name}: on {x.device}, device {dev} expected")
    if not x.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")
    return x.data_ptr()


def _rows_at(x, name, dtype, tokens, heads, d, dev):
    """Pointer and row stride of packed rows: [tokens, heads, d] (or [tokens,
    heads * d]), each token's values in one piece, any distance apart."""
    if x is None or x.__class__ is int:
        return x, 0
    shape = x.shape
    three = len(shape) == 3
    if three:
        ok = shape[1] == heads and shape[2] == d
    else:
        ok = len(shape) == 2 and shape[1] == heads * d
    if ok and x.dtype is dtype and shape[0] >= tokens and x.get_device() == dev:
        if x.is_contiguous():
            return x.data_ptr(), 0
        stride = x.stride()
        if stride[-1] == 1 and (not three or heads == 1 or stride[1] == d):
            if shape[0] == 1:  # a single row's stride says nothing: torch may report any value
                return x.data_ptr(), 0
            if stride[0] >= heads * d:  # (less: rows that overlap, or one row broadcast)
                return x.data_ptr(), stride[0]
    if x.dtype != dtype:
        raise ValueError(f"{name}: dtype {x.dtype}, {dtype} expected")
    if ok and shape[0] >= tokens and x.get_device() != dev:
        raise ValueError(f"{name}: on {x.device}, device {dev} expected")
    raise ValueError(f"{name}: {tuple(shape)} with strides {x.stride()}, [{tokens}, {heads}, {d}] "
                     f"with every token's row in one piece expected")


def _ws_at(x, ws_bytes, dev):
    if x is None or x.__class__ is int:
        return x, int(ws_bytes)
    have = x.numel() * x.element_size()
    if ws_bytes is not None and int(ws_bytes) > have:
        raise ValueError(f"workspace: {have} bytes, ws_bytes = {int(ws_bytes)}")
    if x.get_device() != dev or not x.is_contiguous():
        raise ValueError(f"workspace: contiguous tensor on device {dev} expected")
    return x.data_ptr(), have if ws_bytes is None else int(ws_bytes)


def _attn_call(where, dev, stream, args):
    """The call on its tensors' device, on that device's current stream unless
    `stream` is given."""
    fn = getattr(_lib or load_library(), where)
    if stream is not None or dev is None:
        stream = _stream(stream)
    if dev is not None and dev < 0:
        raise ValueError("device tensor expected")
    if dev is None or dev == _current_device():
        st = fn(*args, _raw_stream(dev) if stream is None else stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev) if stream is None else stream)
    if st:
        raise GDNError(st, where)


def _front_args(cfg, qkv, q_w, k_w, inv_freq, cu_seqlens, kv_lens, t, dev):
    d = cfg.d
    p, row = _rows_at(qkv, "qkv", t, cfg.t_max, cfg.h + 2 * cfg.hkv, d, dev)
    f32, i32, n = torch.float32, torch.int32, cfg.n_max
    return (ctypes.byref(cfg), p, row, _at(q_w, "q_w", f32, d, dev), _at(k_w, "k_w", f32, d, dev),
            _at(inv_freq, "inv_freq", f32, cfg.rot_dim // 2, dev),
            _at(cu_seqlens, "cu_seqlens", i32, n + 1, dev), _at(kv_lens, "kv_lens", i32, n, dev))


def gdn_qk_norm_rope(cfg, qkv, q_w, k_w, inv_freq, cu_seqlens, kv_lens, q, k, stream=None):
    """RMS norm of every query and key head and rotation by the token's position.
    qkv [t_max, (h + 2 hkv) d] may have any row stride (a multiple of 8)."""
    dev, t, d = _dev(qkv, q, k), _GDN_DTYPE.get(cfg.dtype), cfg.d
    n = cfg.t_max * d
    _attn_call("gdn_qk_norm_rope", dev, stream,
               _front_args(cfg, qkv, q_w, k_w, inv_freq, cu_seqlens, kv_lens, t, dev) +
               (_at(q, "q", t, n * cfg.h, dev, d), _at(k, "k", t, n * cfg.hkv, dev, d)))


def gdn_kv_append(cfg, qkv, q_w, k_w, inv_freq, cu_seqlens, kv_lens, block_table, q, k, k_pages,
                  v_pages, stream=None):
    """gdn_qk_norm_rope that also writes k and v into the pages of the cache; q and
    k may be None."""
    dev, t, d, cols, hkv = _dev(qkv, k_pages), _GDN_DTYPE.get(cfg.dtype), cfg.d, cfg.max_pages, cfg.hkv
    n, pool = cfg.t_max * d, cfg.n_pages * hkv * cfg.page_size * d
    _attn_call("gdn_kv_append", dev, stream,
               _front_args(cfg, qkv, q_w, k_w, inv_freq, cu_seqlens, kv_lens, t, dev) +
               (_at(block_table, "block_table", torch.int32, cfg.n_max * cols, dev, cols),
                _at(q, "q", t, n * cfg.h, dev, d), _at(k, "k", t, n * hkv, dev, d),
                _at(k_pages, "k_pages", t, pool, dev, d), _at(v_pages, "v_pages", t, pool, dev, d)))


def gdn_attn_prefill(cfg, q, k, v, cu_q, cu_k, o, workspace, ws_bytes=None, stream=None):
    """Causal attention over packed prompts; q, k, v [tokens, heads, d] may have any
    row stride (a multiple of 8); cu_k None = cu_q."""
    dev, t, i32 = _dev(q, k, v, o), _GDN_DTYPE.get(cfg.dtype), torch.int32
    d, h, hkv, tq, n = cfg.d, cfg.h, cfg.hkv, cfg.t_max, cfg.n_max + 1
    tk = cfg.tk_max or tq
    q, q_row = _rows_at(q, "q", t, tq, h, d, dev)
    k, k_row = _rows_at(k, "k", t, tk, hkv, d, dev)
    v, v_row = _rows_at(v, "v", t, tk, hkv, d, dev)
    ws, ws_bytes = _ws_at(workspace, ws_bytes, dev)
    _attn_call("gdn_attn_prefill", dev, stream,
               (ctypes.byref(cfg), q, q_row, k, k_row, v, v_row, _at(cu_q, "cu_q", i32, n, dev),
                _at(cu_k, "cu_k", i32, n, dev), _at(o, "o", t, tq * h * d, dev, d), ws, ws_bytes))


def gdn_attn_paged(cfg, q, k_pages, v_pages, cu_seqlens, kv_lens, block_table, shared_len, o,
                   workspace, ws_bytes=None, stream=None):
    """Attention of each sequence's new tokens to the pages of the cache; shared_len
    (int32 [1] on the device, or None) positions lie in the same pages for all."""
    dev, t, i32 = _dev(q, k_pages, v_pages, o), _GDN_DTYPE.get(cfg.dtype), torch.int32
    d, h, tq, n, cols = cfg.d, cfg.h, cfg.t_max, cfg.n_max, cfg.max_pages
    pool = cfg.n_pages * cfg.hkv * cfg.page_size * d
    q, q_row = _rows_at(q, "q", t, tq, h, d, dev)
    ws, ws_bytes = _ws_at(workspace, ws_bytes, dev)
    _attn_call("gdn_attn_paged", dev, stream,
               (ctypes.byref(cfg), q, q_row, _at(k_pages, "k_pages", t, pool, dev, d),
                _at(v_pages, "v_pages", t, pool, dev, d),
                _at(cu_seqlens, "cu_seqlens", i32, n + 1, dev),
                _at(kv_lens, "kv_lens", i32, n, dev),
                _at(block_table, "block_table", i32, n * cols, dev, cols),
                _at(shared_len, "shared_len", i32, 1, dev), _at(o, "o", t, tq * h * d, dev, d), ws,
                ws_bytes))


def rope_inv_freq(rot_dim, base=10000.0, factor=1.0, original_len=None, low_turns=1.0,
                  high_turns=32.0, device=None):
    """Radians per position of each pair, fp32 [rot_dim / 2]: base^(-2 i / rot_dim).

    factor > 1 stretches positions for contexts `factor` times longer than the
    model was trained on: without original_len every frequency is divided by it;
    with original_len (the trained length) a pair that makes at least high_turns
    turns over it keeps its frequency, one that makes at most low_turns is
    divided, and those between are blended linearly in the number of turns.
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rot_dim {rot_dim}: an even number expected")
    if not factor > 0 or not base > 0:
        raise ValueError(f"base {base}, factor {factor}: positive numbers expected")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    f = float(base) ** (-2.0 * i / max(rot_dim, 1))
    if original_len is None:
        f = f / factor
    else:
        if not high_turns > low_turns:
            raise ValueError(f"high_turns {high_turns}: more than low_turns {low_turns} expected")
        turns = original_len * f / (2.0 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f.float().to(device) if device is not None else f.float()


def _packed_qkv(qkv, heads, kv_heads):
    if qkv.dim() != 2 or qkv.shape[1] % (heads + 2 * kv_heads):
        raise ValueError(f"qkv [T, ({heads} + 2 * {kv_heads}) * d] expected: {tuple(qkv.shape)}")
    return qkv.shape[0], qkv.shape[1] // (heads + 2 * kv_heads)


def qk_norm_rope(qkv, heads, kv_heads, cu_seqlens, q_weight=None, k_weight=None, inv_freq=None,
                 kv_lens=None, eps=1e-6, interleaved=False, rot_scale=1.0):
    """Allocate outputs with torch and run gdn_qk_norm_rope on the current stream.

    qkv [T, (heads + 2 kv_heads) d] bf16 or fp16; weights fp32 [d] or None (no
    norm); inv_freq fp32 [rot_dim / 2] or None (no rotation); rot_scale a factor
    on cos and sin (0 counts as 1). Returns (q [T, heads, d], k [T, kv_heads,
    d]); v is qkv's last kv_heads d columns."""
    T, d = _packed_qkv(qkv, heads, kv_heads)
    cfg = make_attn_config(T, cu_seqlens.numel() - 1, heads, kv_heads, d, qkv.dtype, eps=eps,
                           rot_dim=0 if inv_freq is None else 2 * inv_freq.numel(),
                           rot_interleaved=interleaved, rot_scale=rot_scale)
    q = torch.empty((T, heads, d), dtype=qkv.dtype, device=qkv.device)
    k = torch.empty((T, kv_heads, d), dtype=qkv.dtype, device=qkv.device)
    if T:
        gdn_qk_norm_rope(cfg, qkv, q_weight, k_weight, inv_freq, cu_seqlens, kv_lens, q, k)
    return q, k


def _pages(k_pages, v_pages, block_table):
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or block_table.dim() != 2:
        raise ValueError(f"k_pages, v_pages [pages, kv_heads, page_size, d] and block_table [N, "
                         f"columns] expected: {tuple(k_pages.shape)}, {tuple(v_pages.shape)}, "
                         f"{tuple(block_table.shape)}")
    return k_pages.shape


def append_paged_kv(qkv, heads, cu_seqlens, kv_lens, block_table, k_pages, v_pages, q_weight=None,
                    k_weight=None, inv_freq=None, eps=1e-6, interleaved=False, rot_scale=1.0,
                    output_k=False):
    """Run gdn_kv_append on the current stream: q and k normed and rotated, k and v
    written into the cache pages of their positions (kv_lens: tokens of each
    sequence in all, these included). Returns q [T, heads, d], or (q, k) with
    output_k."""
    pages, hkv, size, d = _pages(k_pages, v_pages, block_table)
    T, dq = _packed_qkv(qkv, heads, hkv)
    if dq != d:
        raise ValueError(f"qkv: head dim {dq}, {d} expected")
    cfg = make_attn_config(T, cu_seqlens.numel() - 1, heads, hkv, d, qkv.dtype, eps=eps,
                           rot_dim=0 if inv_freq is None else 2 * inv_freq.numel(),
                           rot_interleaved=interleaved, rot_scale=rot_scale, page_size=size,
                           n_pages=pages, max_pages=block_table.shape[1])
    q = torch.empty((T, heads, d), dtype=qkv.dtype, device=qkv.device)
    k = torch.empty((T, hkv, d), dtype=qkv.dtype, device=qkv.device) if output_k else None
    if T:
        gdn_kv_append(cfg, qkv, q_weight, k_weight, inv_freq, cu_seqlens, kv_lens, block_table, q,
                      k, k_pages, v_pages)
    return (q, k) if output_k else q


def _attn_workspace(cfg, device, workspace):
    if workspace is not None:
        return workspace
    with torch.cuda.device(device):
        return torch.empty(gdn_attn_workspace_size(cfg), dtype=torch.uint8, device=device)


def _scale(scale):
    """A caller's score scale (None: the default, which a cfg holds as 0)."""
    if scale is None:
        return 0.0
    if not ctypes.c_float(scale).value > 0.0:
        raise ValueError(f"scale {scale}: a positive number expected")
    return scale


def causal_attention(q, k, v, cu_seqlens, cu_seqlens_k=None, scale=None, workspace=None):
    """Allocate the output with torch and run gdn_attn_prefill on the current stream.

    q [T, heads, d], k and v [Tk, kv_heads, d], bf16 or fp16, rows of any stride;
    the queries are the last tokens of their keys (cu_seqlens_k None: the same
    tokens); scale: of the scores, positive (None: 1 / sqrt(d)). Returns o [T,
    heads, d]; rows that see no key are zeros (k and v may have no row at all), rows
    behind the last sequence are not written."""
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or k.shape[2] != q.shape[2] or \
            not q.dtype == k.dtype == v.dtype:
        raise ValueError(f"q [T, heads, d] and k, v [Tk, kv_heads, d] of one dtype expected: "
                         f"{tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    if cu_seqlens_k is not None and cu_seqlens_k.numel() != cu_seqlens.numel():
        raise ValueError("cu_seqlens and cu_seqlens_k: the same number of sequences expected")
    T, H, d = q.shape
    if cu_seqlens_k is None and k.shape[0] < T:
        raise ValueError(f"k, v: {k.shape[0]} rows, at least {T} expected")
    if k.shape[0] == 0:  # a row that no sequence has (tk_max = 0 would stand for T rows)
        k = v = k.new_zeros((1, *k.shape[1:]))
    cfg = make_attn_config(T, cu_seqlens.numel() - 1, H, k.shape[1], d, q.dtype, _scale(scale),
                           tk_max=k.shape[0])
    o = torch.empty((T, H, d), dtype=q.dtype, device=q.device)
    if T == 0:
        return o
    workspace = _attn_workspace(cfg, q.device, workspace)
    gdn_attn_prefill(cfg, q, k, v, cu_seqlens, cu_seqlens_k, o, workspace)
    return o


def paged_attention(q, k_pages, v_pages, cu_seqlens, kv_lens, block_table, shared_len=None,
                    scale=None, workspace=None, shared_max=None):
    """Allocate the output with torch and run gdn_attn_paged on the current stream.

    q [T, heads, d]: the new tokens of every sequence (one each when decoding),
    whose keys and values the cache already holds; shared_len: int32 [1] on the
    device, positions that lie in the same pages for the whole batch (at most
    shared_max, by default the table's capacity; read once for all where that saves
    more than it costs). Returns o [T, heads, d]."""
    pages, hkv, size, d = _pages(k_pages, v_pages, block_table)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q [T, heads, {d}] expected: {tuple(q.shape)}")
    cols = block_table.shape[1]
    cfg = make_attn_config(q.shape[0], cu_seqlens.numel() - 1, q.shape[1], hkv, d, q.dtype,
                           _scale(scale), page_size=size, n_pages=pages, max_pages=cols,
                           shared_max=0 if shared_len is None else
                           cols * size if shared_max is None else shared_max)
    o = torch.empty((q.shape[0], q.shape[1], d), dtype=q.dtype, device=q.device)
    if q.shape[0] == 0:
        return o
    workspace = _attn_workspace(cfg, q.device, workspace)
    gdn_attn_paged(cfg, q, k_pages, v_pages, cu_seqlens, kv_lens, block_table, shared_len, o,
                   workspace)
    return o
