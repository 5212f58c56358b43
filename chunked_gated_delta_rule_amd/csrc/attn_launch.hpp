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
  // positions of several axes [n_axes][t_max] (null: the place in the sequence), and the
  // axis of each pair
  const int32_t *positions, *pair_axis;
  int n_axes;
  void *q, *k, *k_pages, *v_pages;  // k_pages null: no cache
  uint8_t *k_scales, *v_scales;     // of an 8-bit cache
  int t_max, n_max, h, hkv;
  int rot_dim;
  float eps, rot_scale;
  int page_shift, n_pages, max_pages;
  // set by the launcher: tokens per work-group, and whether the outputs are too large for
  // any cache
  int tokens;
  bool past_cache;
  // 8-bit cache: work-groups per block of tokens, and how many blocks are numbered together
  int parts, group;
};
hipError_t launch_attn_front(const gdn_attn_config *cfg, FrontArgs a, hipStream_t stream);
// The same into an 8-bit cache.
hipError_t launch_attn_append8(const gdn_attn_config *cfg, FrontArgs a, hipStream_t stream);

// A batch whose keys and values lie in pages.
struct PagedBatch {
  const int32_t *cu, *kv_lens, *table, *shared_len;  // shared_len may be null
  int t_max, n_max, page_shift, n_pages, max_pages, shared_max;
};

// Where a tile kernel's keys are: rows of k and v; the pages of each sequence; or
// the pages that the batch shares, for all its tokens at once.
enum class Keys { kRows = 0, kPages = 1, kShared = 2 };

struct TileArgs {
  const void *q, *k, *v;          // k, v: rows, or the page pools
  const uint8_t *k_scales, *v_scales;  // not null: the pools hold 8-bit codes
  int64_t q_row, k_row, v_row;    // elements
  const int32_t *cu_q, *cu_k;     // cu_k: with rows only
  PagedBatch pg;                  // with pages only
  void *o;
  int t_max, tk_max, n_max, h, hkv;
  float scale_log2;               // score scale * log2(e)
  // partial results of keys split over work-groups: [item][split][row]
  float *part_o, *part_ml;
  // filled in by the launcher (TileShape)
  int share, splits, slots, by_keys;
};

// How a call is cut into tiles: rows per tile are tokens times `share` query heads
// of one key head, tt tokens; `slots` token tiles at most, times h / share head
// groups; each tile's keys in `splits` parts. `rows` rows (tt * share, rounded up). by_keys (0:
// not): parts in proportion to the sequences' keys instead, so many work-groups for each head
// group.
struct TileShape {
  int waves, rows, share, tt, slots, splits, by_keys;
};
TileShape tile_shape(const gdn_attn_config *cfg, Keys keys, bool k8);
// Rows of partial results the shape needs (0 where o is written at once).
int64_t tile_part_rows(const gdn_attn_config *cfg, const TileShape &s, Keys keys);
// With more than one split, kRows and kPages are joined into o; the parts of
// kShared are left to the caller.
hipError_t launch_attn_tiles(const gdn_attn_config *cfg, Keys keys, TileArgs a, hipStream_t stream);

struct StreamArgs {
  const void *q;
  int64_t q_row;  // elements
  const void *k_pages, *v_pages;
  const uint8_t *k_scales, *v_scales;  // not null: the pages hold 8-bit codes
  PagedBatch pg;
  void *o;
  int h, hkv;
  float scale_log2;
  int grid;  // work-groups of the main kernel
  // workspace: the prefix's length, and (for tests) whether the keys behind it are read past
  // the caches; 16 bytes per row for the join; the partial results of items split over
  // work-groups (two per work-group); with a shared prefix, the results of items that one
  // work-group finished (one per row) and the prefix's parts
  int32_t *prefix;
  void *plan;
  float *part_o, *part_ml, *done_o, *done_ml;
  const float *pre_o, *pre_ml;
  int pre_share, pre_tt, pre_slots, pre_splits, pre_rows;
};
// Rows (16-row tiles times this) of q that one streamed work item takes.
int stream_row_tiles(const gdn_attn_config *cfg);
// Work-groups of the streaming kernel on the current device.
int stream_grid(const gdn_attn_config *cfg);
// Whether gdn_attn_paged (k8: gdn_attn_paged8) reads a shared prefix once for the whole batch.
bool shares(const gdn_attn_config *cfg, bool k8);
// Whether it streams the keys past few rows, or tiles many rows.
bool streams(const gdn_attn_config *cfg, bool k8);
hipError_t launch_attn_stream(const gdn_attn_config *cfg, StreamArgs a, hipStream_t stream);

}  // namespace gdn
