// C ABI of the softmax-attention operators (declared in include/gdn.h). As in
// gdn_api.cpp every argument is checked on the host before anything is queued;
// nothing here allocates, frees or synchronises.
#include "gdn.h"

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "attn_launch.hpp"

namespace {

constexpr int kMaxHeads = 4096;
constexpr size_t kAlign = 256;
constexpr int kPlanBytes = 16;  // per row
constexpr double kLog2e = 1.4426950408889634;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

gdn_status check_config(const gdn_attn_config *cfg) {
  if (!cfg) return GDN_ERR_INVALID_ARG;
  if (cfg->t_max < 0 || cfg->n_max < 1 || cfg->h < 1 || cfg->hkv < 1) return GDN_ERR_INVALID_ARG;
  if (cfg->dtype != GDN_BF16 && cfg->dtype != GDN_F32 && cfg->dtype != GDN_F16)
    return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(cfg->scale) || !std::isfinite(cfg->rot_scale) || !std::isfinite(cfg->eps) ||
      cfg->eps < 0.f)
    return GDN_ERR_INVALID_ARG;
  if (cfg->scale * kLog2e > FLT_MAX) return GDN_ERR_INVALID_ARG;  // scale_log2, in fp32
  if (cfg->rot_dim < 0 || cfg->rot_dim > cfg->d || cfg->rot_dim % 2 != 0)
    return GDN_ERR_INVALID_ARG;
  if (cfg->rot_interleaved != 0 && cfg->rot_interleaved != 1) return GDN_ERR_INVALID_ARG;
  if (cfg->n_pages < 0 || cfg->max_pages < 0 || cfg->tk_max < 0 || cfg->shared_max < 0)
    return GDN_ERR_INVALID_ARG;
  if (cfg->d != 128 && cfg->d != 256) return GDN_ERR_UNSUPPORTED;
  if (cfg->dtype == GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (cfg->h % cfg->hkv != 0) return GDN_ERR_UNSUPPORTED;
  if (cfg->page_size != 16 && cfg->page_size != 32 && cfg->page_size != 64 &&
      cfg->page_size != 128 && cfg->page_size != 256)
    return GDN_ERR_UNSUPPORTED;
  // positions, and rows of heads, are counted in 32 bits
  if (cfg->t_max > GDN_T_MAX_LIMIT || cfg->tk_max > GDN_T_MAX_LIMIT ||
      cfg->n_max > GDN_N_MAX_LIMIT || cfg->h > kMaxHeads ||
      static_cast<int64_t>(cfg->max_pages) * cfg->page_size > (1 << 30) ||
      static_cast<int64_t>(cfg->t_max) * cfg->h > 0x7fff0000LL)
    return GDN_ERR_CAPACITY;
  return GDN_OK;
}

int page_shift(const gdn_attn_config *cfg) {
  int s = 4;
  while ((1 << s) < cfg->page_size) ++s;
  return s;
}

// What gdn_attn_prefill needs, and what gdn_attn_paged needs, from offset 0 each (a
// workspace serves one call at a time).
struct PrefillLayout {
  size_t part_o, part_ml, total;
};
struct PagedLayout {
  size_t prefix, plan, part_o, part_ml, done_o, done_ml, pre_o, pre_ml, total;
};

struct Taker {
  size_t at = 0;
  size_t operator()(size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  }
};

PrefillLayout prefill_layout(const gdn_attn_config *cfg, gdn::Keys keys, bool k8) {
  const size_t rows = static_cast<size_t>(gdn::tile_part_rows(cfg, gdn::tile_shape(cfg, keys, k8), keys));
  Taker take;
  PrefillLayout l;
  l.part_o = take(rows * cfg->d * 4);
  l.part_ml = take(rows * 2 * 4);
  l.total = take.at;
  return l;
}

PagedLayout paged_layout(const gdn_attn_config *cfg, bool k8) {
  const size_t d = static_cast<size_t>(cfg->d);
  const size_t slots = static_cast<size_t>(gdn::stream_grid(cfg)) * 2 * 16 * gdn::stream_row_tiles(cfg);
  const bool shared = gdn::shares(cfg, k8);
  const size_t done = shared ? static_cast<size_t>(cfg->t_max) * static_cast<size_t>(cfg->h) : 0;
  const size_t pre = shared ? static_cast<size_t>(gdn::tile_part_rows(
                                  cfg, gdn::tile_shape(cfg, gdn::Keys::kShared, k8), gdn::Keys::kShared))
                            : 0;
  Taker take;
  PagedLayout l;
  l.prefix = take(2 * sizeof(int32_t));
  l.plan = take(static_cast<size_t>(cfg->t_max) * cfg->h * kPlanBytes);
  l.part_o = take(slots * d * 4);
  l.part_ml = take(slots * 2 * 4);
  l.done_o = take(done * d * 4);
  l.done_ml = take(done * 2 * 4);
  l.pre_o = take(pre * d * 4);
  l.pre_ml = take(pre * 2 * 4);
  l.total = take.at;
  return l;
}

size_t paged_bytes(const gdn_attn_config *cfg, bool k8) {
  const size_t paged = gdn::streams(cfg, k8) ? paged_layout(cfg, k8).total
                                         : prefill_layout(cfg, gdn::Keys::kPages, k8).total;
  return paged > kAlign ? paged : kAlign;
}

size_t workspace_bytes(const gdn_attn_config *cfg) {
  const size_t prefill = prefill_layout(cfg, gdn::Keys::kRows, false).total, paged = paged_bytes(cfg, false);
  return prefill > paged ? prefill : paged;
}

gdn_status check_workspace(size_t need, const void *ws, size_t bytes) {
  if (!ws || bytes < need || !aligned(ws, kAlign)) return GDN_ERR_WORKSPACE;
  return GDN_OK;
}

// A row stride in elements: 0 = dense; else at least one row, 16-byte steps, and
// at most what lets 64 rows be indexed in 32 bits.
constexpr int64_t kMaxRow = 1 << 24;
bool row_of(int64_t given, int64_t dense, int64_t &row) {
  row = given == 0 ? dense : given;
  return row >= dense && row % 8 == 0 && row <= kMaxRow;
}

float scale_log2(const gdn_attn_config *cfg) {
  const double s = cfg->scale > 0.f ? cfg->scale : 1.0 / std::sqrt(static_cast<double>(cfg->d));
  return static_cast<float>(s * kLog2e);
}

gdn_status from_hip(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }
hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

void tile_common(const gdn_attn_config *cfg, gdn::TileArgs &a, char *ws, size_t part_o,
                 size_t part_ml) {
  a.t_max = cfg->t_max;
  a.n_max = cfg->n_max;
  a.h = cfg->h;
  a.hkv = cfg->hkv;
  a.scale_log2 = scale_log2(cfg);
  a.part_o = reinterpret_cast<float *>(ws + part_o);
  a.part_ml = reinterpret_cast<float *>(ws + part_ml);
}

// Positions of several axes (null: none).
struct Axes {
  const int32_t *positions, *pair_axis;
  int32_t n_axes;
};
// A cache that k and v are written to (null pages: none; null scales: 16-bit).
struct Cache {
  const int32_t *kv_lens, *block_table;
  void *k_pages, *v_pages;
  uint8_t *k_scales, *v_scales;
};

gdn_status front(const gdn_attn_config *cfg, const void *qkv, int64_t qkv_row, const float *q_w,
                 const float *k_w, const float *inv_freq, const Axes &axes,
                 const int32_t *cu_seqlens, const Cache &cache, void *q, void *k, void *stream) {
  if (!qkv || !cu_seqlens || (inv_freq != nullptr) != (cfg->rot_dim > 0))
    return GDN_ERR_INVALID_ARG;
  if (cache.k_pages && (cfg->n_pages < 1 || cfg->max_pages < 1)) return GDN_ERR_INVALID_ARG;
  gdn::FrontArgs a;
  if (!row_of(qkv_row, (static_cast<int64_t>(cfg->h) + 2 * cfg->hkv) * cfg->d, a.qkv_row))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(cache.k_pages, 16) ||
      !aligned(cache.v_pages, 16) || !aligned(q_w, 4) || !aligned(k_w, 4) || !aligned(inv_freq, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(cache.kv_lens, 4) || !aligned(cache.block_table, 4) ||
      !aligned(axes.positions, 4) || !aligned(axes.pair_axis, 4))
    return GDN_ERR_INVALID_ARG;
  a.qkv = qkv;
  a.q_w = q_w;
  a.k_w = k_w;
  a.inv_freq = inv_freq;
  a.cu = cu_seqlens;
  a.kv_lens = cache.kv_lens;
  a.table = cache.block_table;
  a.positions = axes.positions;
  a.pair_axis = axes.pair_axis;
  a.n_axes = axes.n_axes;
  a.q = q;
  a.k = k;
  a.k_pages = cache.k_pages;
  a.v_pages = cache.v_pages;
  a.k_scales = cache.k_scales;
  a.v_scales = cache.v_scales;
  a.t_max = cfg->t_max;
  a.n_max = cfg->n_max;
  a.h = cfg->h;
  a.hkv = cfg->hkv;
  a.rot_dim = cfg->rot_dim;
  a.eps = cfg->eps;
  a.rot_scale = cfg->rot_scale == 0.f ? 1.f : cfg->rot_scale;
  a.page_shift = page_shift(cfg);
  a.n_pages = cfg->n_pages;
  a.max_pages = cfg->max_pages;
  return from_hip(a.k_scales ? gdn::launch_attn_append8(cfg, a, as_stream(stream))
                             : gdn::launch_attn_front(cfg, a, as_stream(stream)));
}

// Axes as a call that needs them takes them.
bool check_axes(const gdn_attn_config *cfg, const Axes &x) {
  return x.positions && x.pair_axis && x.n_axes >= 1 && x.n_axes <= GDN_AXES_LIMIT && cfg->rot_dim > 0;
}

gdn_status paged(const gdn_attn_config *cfg, const void *q, int64_t q_row, const void *k_pages,
                 const void *v_pages, const uint8_t *k_scales, const uint8_t *v_scales,
                 const int32_t *cu_seqlens, const int32_t *kv_lens, const int32_t *block_table,
                 const int32_t *shared_len, void *o, void *workspace, size_t need, size_t ws_bytes,
                 void *stream) {
  if (!q || !k_pages || !v_pages || !cu_seqlens || !kv_lens || !block_table || !o)
    return GDN_ERR_INVALID_ARG;
  if (cfg->n_pages < 1 || cfg->max_pages < 1) return GDN_ERR_INVALID_ARG;
  const gdn_status ws = check_workspace(need, workspace, ws_bytes);
  if (ws != GDN_OK) return ws;
  int64_t row;
  if (!row_of(q_row, static_cast<int64_t>(cfg->h) * cfg->d, row)) return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) ||
      !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4) ||
      !aligned(shared_len, 4))
    return GDN_ERR_INVALID_ARG;
  const bool k8 = k_scales != nullptr;
  char *at = static_cast<char *>(workspace);
  gdn::PagedBatch pg;
  pg.cu = cu_seqlens;
  pg.kv_lens = kv_lens;
  pg.table = block_table;
  pg.shared_len = gdn::shares(cfg, k8) ? shared_len : nullptr;
  pg.t_max = cfg->t_max;
  pg.n_max = cfg->n_max;
  pg.page_shift = page_shift(cfg);
  pg.n_pages = cfg->n_pages;
  pg.max_pages = cfg->max_pages;
  pg.shared_max = cfg->shared_max;
  gdn::TileArgs t = {};
  t.q = q;
  t.q_row = row;
  t.k = k_pages;
  t.v = v_pages;
  t.k_scales = k_scales;
  t.v_scales = v_scales;
  t.cu_q = cu_seqlens;
  t.pg = pg;
  t.o = o;
  if (!gdn::streams(cfg, k8)) {
    const PrefillLayout l = prefill_layout(cfg, gdn::Keys::kPages, k8);
    tile_common(cfg, t, at, l.part_o, l.part_ml);
    return from_hip(gdn::launch_attn_tiles(cfg, gdn::Keys::kPages, t, as_stream(stream)));
  }
  const PagedLayout l = paged_layout(cfg, k8);
  gdn::StreamArgs a = {};
  if (pg.shared_len) {
    tile_common(cfg, t, at, l.pre_o, l.pre_ml);
    const hipError_t e = gdn::launch_attn_tiles(cfg, gdn::Keys::kShared, t, as_stream(stream));
    if (e != hipSuccess) return GDN_ERR_HIP;
    const gdn::TileShape s = gdn::tile_shape(cfg, gdn::Keys::kShared, k8);
    a.pre_share = s.share;
    a.pre_tt = s.tt;
    a.pre_slots = s.slots;
    a.pre_splits = s.splits;
    a.pre_rows = s.rows;
  } else {
    a.pre_share = a.pre_tt = 1;  // the prefix is empty: these are divided by, not used
  }
  a.q = q;
  a.q_row = row;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.pg = pg;
  a.o = o;
  a.h = cfg->h;
  a.hkv = cfg->hkv;
  a.scale_log2 = scale_log2(cfg);
  a.grid = gdn::stream_grid(cfg);
  a.prefix = reinterpret_cast<int32_t *>(at + l.prefix);
  a.plan = at + l.plan;
  a.part_o = reinterpret_cast<float *>(at + l.part_o);
  a.part_ml = reinterpret_cast<float *>(at + l.part_ml);
  a.done_o = reinterpret_cast<float *>(at + l.done_o);
  a.done_ml = reinterpret_cast<float *>(at + l.done_ml);
  a.pre_o = reinterpret_cast<float *>(at + l.pre_o);
  a.pre_ml = reinterpret_cast<float *>(at + l.pre_ml);
  return from_hip(gdn::launch_attn_stream(cfg, a, as_stream(stream)));
}

}  // namespace

extern "C" {

gdn_status gdn_attn_workspace_size(const gdn_attn_config *cfg, size_t *bytes) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  if (!bytes) return GDN_ERR_INVALID_ARG;
  *bytes = workspace_bytes(cfg);
  return GDN_OK;
}

gdn_status gdn_qk_norm_rope(const gdn_attn_config *cfg, const void *qkv, int64_t qkv_row,
                            const float *q_w, const float *k_w, const float *inv_freq,
                            const int32_t *cu_seqlens, const int32_t *kv_lens, void *q, void *k,
                            void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  if (!q || !k) return GDN_ERR_INVALID_ARG;
  return front(cfg, qkv, qkv_row, q_w, k_w, inv_freq, {}, cu_seqlens, {kv_lens}, q, k, stream);
}

gdn_status gdn_qk_norm_rope_axes(const gdn_attn_config *cfg, const void *qkv, int64_t qkv_row,
                                 const float *q_w, const float *k_w, const float *inv_freq,
                                 const int32_t *positions, const int32_t *pair_axis, int32_t n_axes,
                                 const int32_t *cu_seqlens, void *q, void *k, void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  const Axes axes = {positions, pair_axis, n_axes};
  if (!q || !k || !check_axes(cfg, axes)) return GDN_ERR_INVALID_ARG;
  return front(cfg, qkv, qkv_row, q_w, k_w, inv_freq, axes, cu_seqlens, {}, q, k, stream);
}

gdn_status gdn_kv_append(const gdn_attn_config *cfg, const void *qkv, int64_t qkv_row,
                         const float *q_w, const float *k_w, const float *inv_freq,
                         const int32_t *cu_seqlens, const int32_t *kv_lens,
                         const int32_t *block_table, void *q, void *k, void *k_pages,
                         void *v_pages, void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  if (!kv_lens || !block_table || !k_pages || !v_pages) return GDN_ERR_INVALID_ARG;
  return front(cfg, qkv, qkv_row, q_w, k_w, inv_freq, {}, cu_seqlens,
               {kv_lens, block_table, k_pages, v_pages}, q, k, stream);
}

gdn_status gdn_kv_append_axes(const gdn_attn_config *cfg, const void *qkv, int64_t qkv_row,
                              const float *q_w, const float *k_w, const float *inv_freq,
                              const int32_t *positions, const int32_t *pair_axis, int32_t n_axes,
                              const int32_t *cu_seqlens, const int32_t *kv_lens,
                              const int32_t *block_table, void *q, void *k, void *k_pages,
                              void *v_pages, void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  const Axes axes = {positions, pair_axis, n_axes};
  if (!kv_lens || !block_table || !k_pages || !v_pages || !check_axes(cfg, axes))
    return GDN_ERR_INVALID_ARG;
  return front(cfg, qkv, qkv_row, q_w, k_w, inv_freq, axes, cu_seqlens,
               {kv_lens, block_table, k_pages, v_pages}, q, k, stream);
}

gdn_status gdn_kv_append8(const gdn_attn_config *cfg, const void *qkv, int64_t qkv_row,
                          const float *q_w, const float *k_w, const float *inv_freq,
                          const int32_t *positions, const int32_t *pair_axis, int32_t n_axes,
                          const int32_t *cu_seqlens, const int32_t *kv_lens,
                          const int32_t *block_table, void *q, void *k, void *k_pages, void *v_pages,
                          uint8_t *k_scales, uint8_t *v_scales, void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  const Axes axes = {positions, pair_axis, n_axes};
  if (!kv_lens || !block_table || !k_pages || !v_pages || !k_scales || !v_scales)
    return GDN_ERR_INVALID_ARG;
  const bool none = !positions && !pair_axis && n_axes == 0;
  if (!none && !check_axes(cfg, axes)) return GDN_ERR_INVALID_ARG;
  return front(cfg, qkv, qkv_row, q_w, k_w, inv_freq, axes, cu_seqlens,
               {kv_lens, block_table, k_pages, v_pages, k_scales, v_scales}, q, k, stream);
}

gdn_status gdn_attn_prefill(const gdn_attn_config *cfg, const void *q, int64_t q_row,
                            const void *k, int64_t k_row, const void *v, int64_t v_row,
                            const int32_t *cu_q, const int32_t *cu_k, void *o, void *workspace,
                            size_t ws_bytes, void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  if (!q || !k || !v || !cu_q || !o) return GDN_ERR_INVALID_ARG;
  const PrefillLayout l = prefill_layout(cfg, gdn::Keys::kRows, false);
  const gdn_status ws = check_workspace(workspace_bytes(cfg), workspace, ws_bytes);
  if (ws != GDN_OK) return ws;
  gdn::TileArgs a = {};
  const int64_t kv = static_cast<int64_t>(cfg->hkv) * cfg->d;
  if (!row_of(q_row, static_cast<int64_t>(cfg->h) * cfg->d, a.q_row) ||
      !row_of(k_row, kv, a.k_row) || !row_of(v_row, kv, a.v_row))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(cu_q, 4) || !aligned(cu_k, 4))
    return GDN_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.cu_q = cu_q;
  a.cu_k = cu_k ? cu_k : cu_q;
  a.o = o;
  a.tk_max = cfg->tk_max > 0 ? cfg->tk_max : cfg->t_max;
  tile_common(cfg, a, static_cast<char *>(workspace), l.part_o, l.part_ml);
  return from_hip(gdn::launch_attn_tiles(cfg, gdn::Keys::kRows, a, as_stream(stream)));
}

gdn_status gdn_attn_paged(const gdn_attn_config *cfg, const void *q, int64_t q_row,
                          const void *k_pages, const void *v_pages, const int32_t *cu_seqlens,
                          const int32_t *kv_lens, const int32_t *block_table,
                          const int32_t *shared_len, void *o, void *workspace, size_t ws_bytes,
                          void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  return paged(cfg, q, q_row, k_pages, v_pages, nullptr, nullptr, cu_seqlens, kv_lens, block_table,
               shared_len, o, workspace, workspace_bytes(cfg), ws_bytes, stream);
}

gdn_status gdn_attn_paged8_workspace_size(const gdn_attn_config *cfg, size_t *bytes) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  if (!bytes) return GDN_ERR_INVALID_ARG;
  *bytes = paged_bytes(cfg, true);
  return GDN_OK;
}

gdn_status gdn_attn_paged8(const gdn_attn_config *cfg, const void *q, int64_t q_row,
                           const void *k_pages, const void *v_pages, const uint8_t *k_scales,
                           const uint8_t *v_scales, const int32_t *cu_seqlens,
                           const int32_t *kv_lens, const int32_t *block_table,
                           const int32_t *shared_len, void *o, void *workspace, size_t ws_bytes,
                           void *stream) {
  const gdn_status st = check_config(cfg);
  if (st != GDN_OK) return st;
  if (!k_scales || !v_scales) return GDN_ERR_INVALID_ARG;
  return paged(cfg, q, q_row, k_pages, v_pages, k_scales, v_scales, cu_seqlens, kv_lens, block_table,
               shared_len, o, workspace, paged_bytes(cfg, true), ws_bytes, stream);
}

}  // extern "C"
