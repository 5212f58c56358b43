// Device-side parts of the kernels that take query rows in tiles of 32 per wave, with the tiles
// of K and V in LDS: copies into LDS (from rows, from pages, and through registers from pages
// of 8-bit codes), the running state of a wave's rows, and its steps over a tile of keys.
#pragma once

#include <type_traits>

#include "attn_common.hpp"
#include "attn_launch.hpp"

namespace gdn {

namespace {

// instruction kinds of __builtin_amdgcn_sched_group_barrier
constexpr int kSchedValu = 0x2, kSchedMfma = 0x8, kSchedLds = 0x100;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A tile in LDS. Tiles are passed in their own address space and indexed in one
// step from their arrays' start: the compiler then sees which array a read is
// from, and does not make it wait for copies in flight into the others.
template <typename T>
using Lds = __attribute__((address_space(3))) T *;

// Transposing read: within each 16-lane group, lane s supplies four elements
// of row (s >> 2), columns 4 (s & 3) .., and lane j receives column j of the
// four rows.
template <typename T>
__device__ __forceinline__ u32x2 tr_read(Lds<T> tile, int at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(tile + at)));
}

// Parts by keys: at most so many of a tile (one per lane of the join), of at least so many keys.
constexpr int kMostParts = 64, kLeastKeys = 256;

// Head group, tile slot and split of a work-group. The last (longest) tiles come
// first. Unsplit, with a multiple of 8 groups, neighbouring groups (which may read
// the same keys) go to one XCD, whose L2 then holds their keys and values; the
// splits are numbered fastest, so that tiles of the same keys share an XCD.
struct Place {
  int group, slot, split;
};
__device__ __forceinline__ Place place(int wg, int groups, int slots, int splits) {
  if (splits > 1) {
    const int i = wg / splits;
    return {i % groups, slots - 1 - i / groups, wg % splits};
  }
  if (groups % 8 == 0) {
    const int per = groups / 8, i = wg >> 3;
    return {(wg & 7) * per + i % per, slots - 1 - i / per, 0};
  }
  return {wg % groups, slots - 1 - wg / groups, 0};
}
// Number of a tile among the partial results.
__device__ __forceinline__ int64_t item_of(int group, int slot, int groups, int slots) {
  return (int64_t)(slots - 1 - slot) * groups + group;
}

template <typename T, int D, int kBN, int kWaves>
struct Tile {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kPass = 1024 * kWaves;            // bytes the waves copy at a time
  static constexpr int kLoads = kBN * kRowBytes / kPass;
  static constexpr int kRowsPerLoad = kPass / kRowBytes;
};
// Chunk (16 bytes) in which row r keeps its chunk c: c ^ swizzle(r). For K, whose
// fragments take one chunk of 32 rows, the rows differ in the low bits; for V,
// whose transposing reads take four neighbouring chunks of four rows, in bits 2, 3.
__device__ __forceinline__ int k_swz(int r) { return r & 15; }
__device__ __forceinline__ int v_swz(int r) { return (r & 3) << 2; }

// Waits for this wave's reads of LDS and copies into it (lgkmcnt(0), vmcnt(0)).
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);
  asm volatile("" ::: "memory");
}
// A barrier that leaves copies issued since wait_lds() in flight (__syncthreads
// would wait for them).
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Copies kBN rows (those of them that the descriptors' ranges hold, zeros for the
// others) straight to LDS: lane l of wave w fills the 16 bytes at kPass i + 1024 w +
// 16 l with the chunk that belongs there. What a wave copies at a time lies in one
// aligned group of 16 rows: these have one set of swizzles, and lie in one page.
// rsrc(i, add): the descriptor of the wave's i-th group, and what to add to offsets.
// kPast: past the caches (not temporal).
template <typename T, int D, int kBN, int kWaves, bool kV, bool kPast, typename F>
__device__ __forceinline__ void fetch(Lds<T> dst, int row_bytes, int lane, int w, F rsrc) {
  typedef Tile<T, D, kBN, kWaves> L;
  static_assert(L::kRowsPerLoad % 8 == 0, "copies start at even halves of a group");
  const int in = 1024 * w + 16 * lane;
  // a lane's offset in its group, for copies that start in the group's first and
  // (copies of 8 rows) second half
  constexpr int kHalves = L::kRowsPerLoad % 16 ? 2 : 1;
  int from[kHalves];
#pragma unroll
  for (int i = 0; i < kHalves; ++i) {
    const int row = (in / L::kRowBytes + 8 * i) & 15;
    const int ch = in % L::kRowBytes / 16 ^ (kV ? v_swz(row) : k_swz(row));
    from[i] = opaque<D == 256>(row * row_bytes + 16 * ch);
  }
#pragma unroll
  for (int i = 0; i < L::kLoads; ++i) {
    int add = 0;
    const rsrc_t r = rsrc(i / kHalves, add);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (Lds<void>)(dst + L::kPass / 2 * i + 512 * w), 16,
                                             from[i % kHalves] + add, 0, 0, kPast ? 2 : 0);
  }
}

// Running state of a wave's 32 query rows, and its two parts of a step over a
// tile of keys.
template <typename T, int D, int kBN, int kReadAhead = D == 128 ? 8 : 4, int kReadAheadV = D == 128 ? 4 : 2>
struct Rows {
  typedef typename Elem<T>::vec8 vec8;
  static constexpr int kT = kBN / 32;
  vec8 q[D / 16];
  f32x16 o[D / 32];
  f32x16 sc[kT];
  float m, l;  // maximum (log2 scale) and this lane's part of the sum
  // weights are 2^(sc * mul - sub): with the scale and the maximum (less kWeightLog2), or with
  // 1 and 0 where some row's maximum is far (past kFarLog2) and score() leaves exponents in sc
  float mul, sub;
  int far;

  __device__ __forceinline__ void load(const T *row, int hh, float scale_log2) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      q[i] = *reinterpret_cast<const vec8 *>(row + 8 * hh + 16 * i);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    m = kNegInf;
    l = 0.f;
    mul = scale_log2;
    sub = -Elem<T>::kWeightLog2;
    far = 0;
  }

  // (not seen through: the compiler would copy the rest of the step for either answer,
  // which costs the part kernel its registers)
  __device__ __forceinline__ bool is_far() const { return uniform(opaque<true>(far)); }

  // Scores of the tile, and the running maximum.
  __device__ __forceinline__ void score(Lds<T> kt, int k0, int lim, bool masked, float scale_log2,
                                        int lane) {
    const int col = lane & 31, hh = lane >> 5;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
    // row col, chunk (2 i + hh) ^ swizzle: rows are multiples of 128 values, so the
    // chunk's changes are bit flips of one address
    const int base = opaque<D == 256>(col * D + 8 * (k_swz(col) ^ hh));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int at = (base ^ (16 * (i & 7))) + 128 * (i >> 3);
#pragma unroll
      for (int t = 0; t < kT; ++t)
        sc[t] = mfma32(*(Lds<const vec8>)(kt + at + 32 * t * D), q[i], sc[t]);
    }
    // order: some fragments ahead (with heads of 256 as many as the registers leave), then
    // products and reads in turn
    constexpr int kAhead = kReadAhead;
    __builtin_amdgcn_sched_group_barrier(kSchedLds, kAhead, 0);
#pragma unroll
    for (int i = 0; i < (D / 16 * kT - kAhead) / 2; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedLds, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, kAhead, 0);
    if (masked) {
      const int last = opaque<true>(lim - k0 - 4 * hh);
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sc[t][i] = 32 * t + 8 * (i >> 2) + (i & 3) <= last ? sc[t][i] : kNegInf;
    }
    float mx = kNegInf;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[t][i]);
    mx = max32(mx) * scale_log2;
    if (__any(mx > m + kRescaleLog2)) {
      const float mn = fmaxf(m, mx);
      const float al = mn == kNegInf ? 1.f : fast_exp2(m - mn);
      m = mn;
      l *= al;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[i][k] *= al;
      const float ms = m == kNegInf ? 0.f : m;
      far = __any(fabsf(ms) > kFarLog2);
      mul = far ? 1.f : scale_log2;
      sub = (far ? 0.f : ms) - Elem<T>::kWeightLog2;
    }
    if (is_far()) {
      const float ms = m == kNegInf ? 0.f : m;
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[t][i] = far_exponent(sc[t][i], scale_log2, ms);
    }
  }

  // Weights of the tile, and their products with its values.
  __device__ __forceinline__ void weigh(Lds<T> vt, float scale_log2, int lane) {
    float by = mul, ms = sub;
    if constexpr (D == 256) {  // (no register left to keep them: 16384 tokens 1900 us against 1805)
      const bool f = is_far();
      by = f ? 1.f : scale_log2;
      ms = (f || m == kNegInf ? 0.f : m) - Elem<T>::kWeightLog2;
    }
    // lane's part of a transposing read: row 4 hh + (s16 >> 2) (+ 8), columns 32 i +
    // 16 gb + 4 (s16 & 3)
    const int hh = lane >> 5, s16 = lane & 15, gb = (lane >> 4) & 1, r0 = 4 * hh + (s16 >> 2);
    const int base =
        opaque<D == 256>(r0 * D + 4 * (s16 & 1) + 8 * (v_swz(r0) ^ (2 * gb + ((s16 & 3) >> 1))));
    // 16 keys at a time: the weights of the next are formed while the products
    // of these run
#pragma unroll
    for (int b = 0; b < 2 * kT; ++b) {
      uint32_t wd[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e0 = fast_exp2(fmaf(sc[b >> 1][8 * (b & 1) + 2 * i], by, -ms));
        const float e1 = fast_exp2(fmaf(sc[b >> 1][8 * (b & 1) + 2 * i + 1], by, -ms));
        l += e0 + e1;
        wd[i] = Elem<T>::pack(e0, e1);
      }
      const vec8 p = __builtin_bit_cast(vec8, u32x4{wd[0], wd[1], wd[2], wd[3]});
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int at = (base ^ (32 * (i & 3))) + 128 * (i >> 2);
        const u32x2 x = tr_read<T>(vt, at + 16 * b * D), y = tr_read<T>(vt, at + (16 * b + 8) * D);
        o[i] = mfma32(__builtin_bit_cast(vec8, u32x4{x[0], x[1], y[0], y[1]}), p, o[i]);
      }
    }
    // order: the first keys' fragments and weights, then under each product the
    // reads of a later one and (heads of 128) a part of the next weights
    constexpr int kAhead = kReadAheadV;
    __builtin_amdgcn_sched_group_barrier(kSchedLds, 2 * kAhead, 1);
    if (D == 128) __builtin_amdgcn_sched_group_barrier(kSchedValu, 28, 1);
#pragma unroll
    for (int i = 0; i < D / 32 * 2 * kT - kAhead; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedLds, 2, 1);
      if (D == 128) __builtin_amdgcn_sched_group_barrier(kSchedValu, 7, 1);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, kAhead, 1);
  }

  // The running state as it is, for a later join.
  __device__ __forceinline__ void store_part(float *po, float *pm, int hh) const {
    const float sum = sum32(l);
    if (hh == 0) *reinterpret_cast<f32x2 *>(pm) = f32x2{m, sum};
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<f32x4 *>(po + 32 * i + 8 * b + 4 * hh) =
            f32x4{o[i][4 * b], o[i][4 * b + 1], o[i][4 * b + 2], o[i][4 * b + 3]};
  }

  __device__ __forceinline__ void store(T *row, int hh) {
    const float sum = sum32(l);
    float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees no key gives zeros
    if constexpr (std::is_same_v<T, _Float16>) {
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(o[i][k]));
      if (__any(most * inv >= kPastF16)) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k) o[i][k] = mean_f16(o[i][k] * inv);
        inv = 1.f;
      }
    }
    // a lane and its partner 32 lanes on hold halves of 8 dims: swapped in pairs of
    // blocks, each lane has 16 bytes in a row
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int b = 0; b < 4; b += 2) {
        uint32_t u[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            u[k][e] = Elem<T>::pack(o[i][4 * (b + k) + 2 * e] * inv, o[i][4 * (b + k) + 2 * e + 1] * inv);
        const auto x0 = __builtin_amdgcn_permlane32_swap(u[0][0], u[1][0], false, false);
        const auto x1 = __builtin_amdgcn_permlane32_swap(u[0][1], u[1][1], false, false);
        if (row)
          *reinterpret_cast<u32x4 *>(row + 32 * i + 8 * b + 8 * hh) = u32x4{x0[0], x1[0], x0[1], x1[1]};
      }
  }
};

// The tile of a work-group: its heads and sequence, the sequence's rows and keys, the
// tile's first token, and the part of its keys.
struct Where {
  int group, slot, split, splits, s, qb, lq, kb, lk, q0, past;
  int past_cache;  // pages read once, and too large in all for the caches
  // one value per wave, which the compiler does not see by itself
  __device__ __forceinline__ Where uniform_() const {
    return {uniform(group), uniform(slot), uniform(split), uniform(splits), uniform(s),  uniform(qb),
            uniform(lq),    uniform(kb),   uniform(lk),    uniform(q0),     uniform(past),
            uniform(past_cache)};
  }
};
// key_bytes: of a key and its value, of one key head.
// kByKeys: the tile's parts go by its sequence's keys (TileArgs::by_keys), and slot is the
// part's number in its head group.
template <Keys kKeys, bool kSplit, int kThreads, bool kByKeys = false>
__device__ __forceinline__ bool find(const TileArgs &a, int tt, int key_bytes, int tid, Where &t,
                                     int (&lds)[kThreads / 64][2]) {
  if constexpr (kByKeys) {
    const int groups = a.h / a.share, wg = flat_block(), lane = tid & 63;
    t.slot = wg / groups;
    t.group = wg - t.slot * groups;
    t.past_cache = 0;
    Tiled p;
    int first;
    auto in = [&](const auto &batch) {
      t.past_cache = batch.past_cache(a.hkv * key_bytes);
      return batch.in_parts(
          lane, a.by_keys, kMostParts, kLeastKeys,
          [&](const Tiled &x, int first, int parts) {
            return t.slot >= first && t.slot < first + (x.n + tt - 1) / tt * parts;
          },
          p, first, t.splits);
    };
    auto keys = [&](int i, int(&o)[2]) {
      o[0] = 0;
      o[1] = kv_of(a.pg, i);
    };
    if (!(a.n_max <= 64 ? in(TiledBatch<1>(a.cu_q, a.n_max, a.t_max, tt, lane, keys))
                        : in(TiledBatch<4>(a.cu_q, a.n_max, a.t_max, tt, lane, keys))))
      return false;
    const int i = t.slot - first, tile = i / t.splits;
    t.split = i - tile * t.splits;
    t.q0 = tile * tt;
    t.s = p.s;
    t.qb = p.b;
    t.lq = p.n;
    t.kb = 0;
    t.lk = p.extra[1];
    t.past = t.lk - t.lq;
    return true;
  }
  const Place at = place(flat_block(), a.h / a.share, a.slots, a.splits);
  t.group = at.group;
  t.slot = at.slot;
  t.split = at.split;
  t.splits = a.splits;
  t.past_cache = 0;
  if (at.slot < 0) return false;  // past the grid's count (last row)
  if constexpr (kKeys == Keys::kShared) {
    const Prefix p = shared_prefix<kThreads>(a.pg, tid, lds);
    t.s = p.seq;
    t.qb = t.kb = 0;
    t.lq = cu_at(a.cu_q, a.n_max, a.t_max);
    t.lk = p.len;
    t.q0 = at.slot * tt;
    t.past = t.lk;  // every token sees the whole prefix
    return t.q0 < t.lq && t.lk > 0;
  } else {
    auto keys = [&](int i, int(&o)[2]) {
      if constexpr (kKeys == Keys::kRows) {
        o[0] = cu_at(a.cu_k, i, a.tk_max);
        o[1] = cu_end(a.cu_k, i, o[0], a.tk_max) - o[0];
      } else {
        o[0] = 0;
        o[1] = kv_of(a.pg, i);
      }
    };
    const int lane = tid & 63, over = a.slots - at.slot;
    Tiled p;
    if constexpr (kSplit) {
      // the batch's tiles, last one first, then the slots that are left over
      int first, total;
      auto in = [&](const auto &batch) {
        if constexpr (kKeys == Keys::kPages) t.past_cache = batch.past_cache(a.hkv * key_bytes);
        return batch.in_order(
            lane,
            [&](const Tiled &x, int first, int total) {
              const int i = min(total, a.slots) - over;
              return i >= first && i < first + (x.n + tt - 1) / tt;
            },
            p, first, total);
      };
      if (!(a.n_max <= 64 ? in(TiledBatch<1>(a.cu_q, a.n_max, a.t_max, tt, lane, keys))
                          : in(TiledBatch<4>(a.cu_q, a.n_max, a.t_max, tt, lane, keys))))
        return false;
      t.slot = min(total, a.slots) - over;
      t.q0 = (t.slot - first) * tt;
    } else if (a.n_max == 1) {
      p.s = 0;
      p.b = cu_at(a.cu_q, 0, a.t_max);
      p.n = cu_end(a.cu_q, 0, p.b, a.t_max) - p.b;
      keys(0, p.extra);
      t.q0 = ((p.n + tt - 1) / tt - over) * tt;
    } else if (a.n_max <= kMostTiled) {
      int tile;
      if (!(a.n_max <= 64 ? TiledBatch<1>(a.cu_q, a.n_max, a.t_max, tt, lane, keys)
                                .longest_first(lane, over - 1, p, tile)
                          : TiledBatch<4>(a.cu_q, a.n_max, a.t_max, tt, lane, keys)
                                .longest_first(lane, over - 1, p, tile)))
        return false;
      t.q0 = tile * tt;
    } else {
      const Packed q = locate(
          a.cu_q, a.n_max, a.t_max, at.slot, lane, [&](int i, int b) { return b / tt + i; }, keys,
          p.extra);
      p.s = q.s;
      p.b = q.b;
      p.n = q.n;
      t.q0 = (at.slot - (p.b / tt + p.s)) * tt;
    }
    t.s = p.s;
    t.qb = p.b;
    t.lq = p.n;
    t.kb = p.extra[0];
    t.lk = p.extra[1];
    t.past = t.lk - t.lq;                  // token r sees keys 0 .. past + r
    return t.q0 >= 0 && t.q0 < t.lq;       // else no tile of the sequence has this slot
  }
}

// What the tile's rows see: keys 0 .. `keys` - 1 some row; lo (hi): the last key that
// the wave's first (last) row sees, lim this lane's row.
struct Sight {
  int tok, lim, lo, hi, keys;
};
// rw: the wave's first row of the tile, tt tokens times `share` heads.
template <Keys kKeys>
__device__ __forceinline__ Sight sight_of(const Where &t, int rw, int col, int tt, int share) {
  Sight s;
  // rows past the tile's tokens or the sequence's end take the last token's limit
  // and are not stored
  s.tok = min(t.q0 + (rw + col) / share, t.lq - 1);
  s.lim = t.past + s.tok;
  s.lo = t.past + min(t.q0 + rw / share, t.lq - 1);
  s.hi = t.past + min(t.q0 + min((rw + 31) / share, tt - 1), t.lq - 1);
  s.keys = min(t.past + min(t.q0 + tt, t.lq), t.lk);
  if constexpr (kKeys == Keys::kShared) {
    s.lim = s.lo = s.hi = t.lk - 1;
    s.keys = t.lk;
  }
  if (t.q0 + rw / share >= t.lq) s.hi = -1;  // none of the wave's rows is the sequence's
  return s;
}

// The pages of the groups of 16 keys that a wave copies of a tile. Looked up a phase
// before the copies, which then start at once.
template <typename L, Keys kKeys>
struct Spot {
  static constexpr int kN = L::kLoads * L::kRowsPerLoad / 16;
  int page[kN];
  // first key of the wave's i-th group in the tile
  static __device__ __forceinline__ int key(int i, int w) {
    return 16 * ((i * (L::kRowsPerLoad < 16 ? 16 : L::kRowsPerLoad) + 1024 / L::kRowBytes * w) / 16);
  }
  __device__ __forceinline__ void look(const TileArgs &a, const Where &t, int k0, int w) {
    if constexpr (kKeys != Keys::kRows) {
#pragma unroll
      for (int i = 0; i < kN; ++i) page[i] = page_of(a.pg, t.s, min(k0 + key(i, w), t.lk - 1));
    }
  }
};

// Copies the kBN keys (values) from k0 on to LDS, as ranges that end with the
// sequence's last key. kWaves waves take part, of which this is number w.
template <typename T, int D, int kBN, int kWaves, Keys kKeys, bool kV, bool kPast = false>
__device__ __forceinline__ void get(const TileArgs &a, const Where &t,
                                    const Spot<Tile<T, D, kBN, kWaves>, kKeys> &spot, int kvh, int k0,
                                    T *tile, int lane, int w) {
  const T *base = static_cast<const T *>(kV ? a.v : a.k);
  if constexpr (kKeys == Keys::kRows) {
    const int64_t stride = kV ? a.v_row : a.k_row;
    const int row_bytes = (int)stride * 2;
    const rsrc_t r = make_rsrc(base + (t.kb + k0) * stride + kvh * D,
                               (min(kBN, t.lk - k0) - 1) * row_bytes + D * 2);
    fetch<T, D, kBN, kWaves, kV, kPast>((Lds<T>)tile, row_bytes, lane, w, [&](int i, int &add) {
      add = spot.key(i, w) * row_bytes;
      return r;
    });
  } else {
    fetch<T, D, kBN, kWaves, kV, kPast>((Lds<T>)tile, D * 2, lane, w, [&](int i, int &) {
      const int key = k0 + spot.key(i, w);
      const T *p = base + pool_row(a.pg, spot.page[i], key, kvh, a.hkv) * D;
      return make_rsrc(p, max(min(16, t.lk - key), 0) * D * 2);
    });
  }
}

// Tiles of an 8-bit cache: the codes of a tile to come wait in registers (ask), and are
// written to LDS as 16-bit values (put) once its place is free, each by one wave for all.
// A lane's 16 codes are 16 dims of a row in a group of 16 keys, which lies in one page and
// has one scale. In registers, as only they can turn codes into values; so each code is
// turned once for the 128 or 256 rows of a tile, and the products read what they read of a
// 16-bit cache. The conversions and the writes (two of 16 bytes per load) cost a full tile
// nothing that is seen with heads of 128 (a chunk of 2048 tokens on 8003 keys, back to back, 256
// us against 255 over 16-bit pages; the first passes after a pause 283 and 285), and a sixth
// with heads of 256 (312 against 268; 362 and 299), whose registers then leave no reads ahead.
// Half the bytes pay where keys are many and rows few (4 sequences of 8 tokens on 43000 keys
// 61 against 80).
template <typename T, int D, int kBN, int kWaves>
struct Codes {
  static constexpr int kPass = 1024 * kWaves;  // bytes the waves load at a time
  static constexpr int kN = kBN * D / kPass;
  static_assert(kN > 0 && kBN * D % kPass == 0 && 16 * D % 1024 == 0, "whole loads, in one group each");
  u32x4 x[kN];
  uint32_t scale[kN];

  // the wave's i-th load: its first byte in the tile, and the group that holds it
  static __device__ __forceinline__ int from(int i, int w) { return kPass * i + 1024 * w; }
  static __device__ __forceinline__ int group(int i, int w) { return from(i, w) / D & ~15; }

  struct Pages {
    int word[kN];
    __device__ __forceinline__ void look(const TileArgs &a, const Where &t, int k0, int w) {
#pragma unroll
      for (int i = 0; i < kN; ++i) word[i] = page_word(a.pg, t.s, max(min(k0 + group(i, w), t.lk - 1), 0));
    }
  };
  // there: whether there is such a tile. The loads are made all the same, of nothing: behind a
  // branch around them the compiler could not count them, and every wait would be for all
  // loads (512 tokens on 8192 keys 95 us against 89). kPast: past the caches.
  template <bool kPast>
  __device__ __forceinline__ void ask(const void *pool, const uint8_t *scales, const TileArgs &a,
                                      const Where &t, const Pages &at, int kvh, int k0, bool there,
                                      int lane, int w) {
    if constexpr (D == 256) lane = fresh_lane();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int key = k0 + group(i, w), last = max(min(key, t.lk - 1), 0);
      const int page = page_in(a.pg, at.word[i]);
      const uint8_t *p = static_cast<const uint8_t *>(pool) + pool_row(a.pg, page, key, kvh, a.hkv) * D;
      // a range that ends with the sequence's last key: zeros past it
      const rsrc_t r = uniform_rsrc(p, there ? max(min(16, t.lk - key), 0) * D : 0);
      x[i] = __builtin_amdgcn_raw_buffer_load_b128(
          r, (from(i, w) - group(i, w) * D) + 16 * lane, 0, kPast ? 2 : 0);
      scale[i] = scales[scale_at(a.pg, page, last, kvh, a.hkv)];
    }
  }
  template <bool kV>
  __device__ __forceinline__ void put(Lds<T> tile, int lane, int w) const {
    if constexpr (D == 256) lane = fresh_lane();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = from(i, w) + 16 * lane, row = at / D, ch = at % D / 8;
      const int swz = kV ? v_swz(row) : k_swz(row);
      const float s = scale_of(scale[i]);
      *(Lds<u32x4>)(tile + row * D + 8 * (ch ^ swz)) = values8<T>(x[i][0], x[i][1], s);
      *(Lds<u32x4>)(tile + row * D + 8 * ((ch + 1) ^ swz)) = values8<T>(x[i][2], x[i][3], s);
    }
  }
};

// How a wave's part of the tiles gets into LDS: copied straight, or (k8) through registers,
// one tile further ahead. to() brings the tile that starts at key k0 (k8: asked for before; it
// then asks for the next one, from k1, whose pages `spot` names); a key below 0: there is none.
template <typename T, int D, int kBN, int kWaves, Keys kKeys, bool k8>
struct Bring {
  static constexpr int kAhead = 0;
  typedef Spot<Tile<T, D, kBN, kWaves>, kKeys> Spots;
  template <bool kV, bool kPast>
  __device__ __forceinline__ void first(const TileArgs &, const Where &, const Spots &, int, int, int, int) {}
  template <bool kV, bool kPast>
  __device__ __forceinline__ void to(T *tile, const TileArgs &a, const Where &t, const Spots &spot,
                                     int kvh, int k0, int, int lane, int w) {
    if (k0 >= 0) get<T, D, kBN, kWaves, kKeys, kV, kPast>(a, t, spot, kvh, k0, tile, lane, w);
  }
};
template <typename T, int D, int kBN, int kWaves, Keys kKeys>
struct Bring<T, D, kBN, kWaves, kKeys, true> {
  static constexpr int kAhead = 1;
  typedef Codes<T, D, kBN, kWaves> Held;
  typedef typename Held::Pages Spots;
  Held k, v;
  template <bool kV, bool kPast>
  __device__ __forceinline__ void first(const TileArgs &a, const Where &t, const Spots &spot, int kvh,
                                        int k0, int lane, int w) {
    if constexpr (kV)
      v.template ask<kPast>(a.v, a.v_scales, a, t, spot, kvh, max(k0, 0), k0 >= 0, lane, w);
    else
      k.template ask<kPast>(a.k, a.k_scales, a, t, spot, kvh, max(k0, 0), k0 >= 0, lane, w);
  }
  template <bool kV, bool kPast>
  __device__ __forceinline__ void to(T *tile, const TileArgs &a, const Where &t, const Spots &spot,
                                     int kvh, int, int k1, int lane, int w) {
    if constexpr (kV)
      v.template put<true>((Lds<T>)tile, lane, w);
    else
      k.template put<false>((Lds<T>)tile, lane, w);
    first<kV, kPast>(a, t, spot, kvh, k1, lane, w);
  }
};
// The wait before a barrier: codes that were asked for go on coming.
template <bool k8>
__device__ __forceinline__ void wait_tiles() {
  if constexpr (k8) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
  } else {
    wait_lds();
  }
}

template <typename T>
__device__ __forceinline__ const T *q_row(const TileArgs &a, const Where &t, int tok, int row, int D) {
  return static_cast<const T *>(a.q) + (int64_t)(t.qb + tok) * a.q_row +
         (t.group * a.share + row % a.share) * D;
}

}  // namespace

}  // namespace gdn
