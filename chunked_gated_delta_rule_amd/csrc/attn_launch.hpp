// Host-side launchers of the softmax-attention kernels (internal to the
// library). Each enqueues work on `stream` and returns the launch status; none
// allocates or synchronises. Shapes have already been validated by the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_launch.hpp"

namespace gdn {

struct FrontArgs {
  const void *qkv;
  int64_t qkv_row;  // elements
  const float *q_w, *k_w, *inv_freq;
  const int32_t *cu, *kv_lens, *table;
  void *q, *k, *k_pages, *v_pages;  // k_pages null: no cache
  int t_max, n_max, h, hkv;
  int rot_dim;
  float eps, rot_scale;
  int page_shift, n_pages, max_pages;
};
hipError_t launch_attn_front(const gdn_attn_config *cfg, FrontArgs a, hipStream_t stream);

struct PrefillArgs {
  const void *q, *k, *v;
  int64_t q_row, k_row, v_row;  // elements
  const int32_t *cu_q, *cu_k;
  void *o;
  int t_max, tk_max, n_max, h, hkv;
  float scale_log2;  // score scale * log2(e)
  int share;         // query heads of one key head that a tile's rows share
};
hipError_t launch_attn_prefill(const gdn_attn_config *cfg, PrefillArgs a, hipStream_t stream);

struct PagedArgs {
  const void *q;
  int64_t q_row;  // elements
  const void *k_pages, *v_pages;
  const int32_t *cu, *kv_lens, *table, *shared_len;
  void *o;
  int t_max, n_max, h, hkv;
  int page_shift, n_pages, max_pages, shared_max;
  float scale_log2;
  int grid;  // work-groups of the main kernel
  // workspace: the plan, the partial results of items split over work-groups
  // (two per work-group), and with a shared prefix the results of items that
  // one work-group finished (two per row: the prefix's and the sequence's)
  int32_t *plan;
  float *part_o, *part_ml, *done_o, *done_ml;
};
// Rows (16-row tiles times this) of q that one paged work item takes.
int paged_row_tiles(const gdn_attn_config *cfg);
// Work-groups of the paged kernel on the current device.
int paged_grid(const gdn_attn_config *cfg);
hipError_t launch_attn_paged(const gdn_attn_config *cfg, PagedArgs a, hipStream_t stream);

}  // namespace gdn
