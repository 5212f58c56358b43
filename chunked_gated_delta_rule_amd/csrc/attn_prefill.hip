// Causal attention over packed prompts (grouped heads, queries the last tokens of their
// keys) and over the pages of a cache, forward:
//   o_r = sum_{c <= lim(r)} softmax_c(scale q_r . k_c) v_c.
//
// One pass over the keys per tile of query rows, with a running maximum and sum per row
// (the maximum moves only when it has grown by 2^8, so the output sums are rarely
// rescaled). A tile's rows are tokens times the query heads that share a key head, 32
// rows per wave; the tiles of K and V go straight to LDS (16-byte copies that pass no
// register), double buffered, and are shared by the waves. Everything else stays in the
// wave's registers: scores are formed transposed, S^T = K Q^T, so a lane's column is
// one query row and the statistics are per lane (one exchange between the half-waves
// per tile), and the C layout of S^T is, with the keys taken in the order the
// accumulator holds them, the B operand of O^T += V^T P^T. V^T comes from the row-major
// tile by transposing LDS reads. So scores and weights never touch LDS.
//
// LDS rows are swizzled by 16-byte chunk: the 32 rows that a K fragment reads at one
// chunk, and the rows that a transposing read spans, fall into different banks (no
// conflict is counted).
//
// Rounding to 16 bits: the weights, for their product with V (by half a step, 2^-8 or 2^-11
// of the weight; fp16 ones below 2^-21 of the row's largest by 2^-32 of that), and the
// output, once. Sums are fp32.
//
// Bound by the matrix instructions and the exponentials between them; long prompts come
// near what a large matrix product reaches: one of 4096 tokens, 32 heads of 128 137 us
// (1.00 PFLOP/s; a product of 8192^3 1.26), one of 16384, 16 heads of 256 1.90 ms (1.16
// PFLOP/s). Boxes differ (133 to 147 us, 1.85 to 1.92 ms), and back to back the card lowers
// its clock (162 us after twenty of the former). Short ones wait for their first keys and
// for each other's copies: 32 of 58 to 1203 tokens 146 us, where bytes and products would
// each take 78. A single prompt of some thousand tokens with few heads is uneven work: its
// tiles see very different numbers of keys (4000 tokens, 16 heads of 128: 99 us against 52).
#include "attn_common.hpp"
#include "attn_launch.hpp"

#include <type_traits>

namespace gdn {

namespace {

constexpr int kPartRows = 128;  // rows of a tile whose keys are split

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
template <typename T, int D, int kBN>
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
    constexpr int kAhead = D == 128 ? 8 : 4;
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
    constexpr int kAhead = D == 128 ? 4 : 2;
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
  int group, slot, split, s, qb, lq, kb, lk, q0, past;
  int past_cache;  // pages read once, and too large in all for the caches
  // one value per wave, which the compiler does not see by itself
  __device__ __forceinline__ Where uniform_() const {
    return {uniform(group), uniform(slot), uniform(split), uniform(s),  uniform(qb),
            uniform(lq),    uniform(kb),   uniform(lk),    uniform(q0), uniform(past),
            uniform(past_cache)};
  }
};
template <int D, Keys kKeys, bool kSplit, int kThreads>
__device__ __forceinline__ bool find(const TileArgs &a, int tt, int tid, Where &t,
                                     int (&lds)[kThreads / 64][2]) {
  const Place at = place(flat_block(), a.h / a.share, a.slots, a.splits);
  t.group = at.group;
  t.slot = at.slot;
  t.split = at.split;
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
        if constexpr (kKeys == Keys::kPages) t.past_cache = batch.past_cache(a.hkv * D * 4);
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

template <typename T>
__device__ __forceinline__ const T *q_row(const TileArgs &a, const Where &t, int tok, int row, int D) {
  return static_cast<const T *>(a.q) + (int64_t)(t.qb + tok) * a.q_row +
         (t.group * a.share + row % a.share) * D;
}

// Whole tiles: kWaves waves of 32 rows. With four (D = 128, shorter sequences), three
// work-groups share a CU and overlap one's start and end with another's products; the
// keys go 32 at a time, for which the registers suffice (two work-groups and 64 keys:
// 128 sequences of 128 tokens 97 us against 85). With eight, the two waves of a SIMD (w
// and w + 4) go through the two parts of a step in opposite order, a barrier after each
// part: while one runs its score products the other forms weights (16384 tokens, 16
// heads of 256: 2658 us with four waves, 2130 with eight, when this was built; now 1900).
// Their steps have 64 keys, or 32 with heads of 256, which leaves registers to read
// fragments ahead (1836 -> 1820).
template <typename T, int D, int kWaves, Keys kKeys>
__global__ __launch_bounds__(64 * kWaves, kWaves == 4 ? 3 : 2) void attn_tile_kernel(TileArgs a) {
  constexpr int kBM = 32 * kWaves, kBN = kWaves == 4 || D == 256 ? 32 : 64;
  // four arrays of their own, so that a tile in flight is known to be another
  // than the ones being read
  __shared__ __attribute__((aligned(16))) T k_a[kBN * D], v_a[kBN * D], k_b[kBN * D], v_b[kBN * D];
  __shared__ int scan[kWaves][2];

  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  Where t;
  const int share = a.share, tt = kBM / share;
  if (!find<D, kKeys, false, 64 * kWaves>(a, tt, tid, t, scan)) return;
  t = t.uniform_();
  const int kvh = t.group * share / (a.h / a.hkv);
  const Sight see = sight_of<kKeys>(t, 32 * w, col, tt, share);
  const int tiles = see.keys > 0 ? (see.keys + kBN - 1) / kBN : 0;

  typedef Spot<Tile<T, D, kBN, kWaves>, kKeys> Spots;
  auto look = [&](int j) __attribute__((always_inline)) {
    Spots s = {};
    if (j < tiles) s.look(a, t, j * kBN, w);
    return s;
  };
  auto get_k = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
    if (j < tiles) get<T, D, kBN, kWaves, kKeys, false>(a, t, s, kvh, j * kBN, tile, lane, w);
  };
  auto get_v = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
    if (j < tiles) get<T, D, kBN, kWaves, kKeys, true>(a, t, s, kvh, j * kBN, tile, lane, w);
  };
  Rows<T, D, kBN> x;
  {
    const Spots s = look(0);
    get_k(0, k_a, s);
    get_v(0, v_a, s);
  }
  x.load(q_row<T>(a, t, see.tok, 32 * w + col, D), hh, a.scale_log2);
  auto score = [&](int j, T *kt) __attribute__((always_inline)) {
    const int k0 = j * kBN;
    if (k0 <= see.hi) x.score((Lds<T>)kt, k0, see.lim, k0 + kBN - 1 > see.lo, a.scale_log2, lane);
  };
  auto weigh = [&](int j, T *vt) __attribute__((always_inline)) {
    if (j * kBN <= see.hi) x.weigh((Lds<T>)vt, a.scale_log2, lane);
  };
  if constexpr (kWaves == 4) {
    Spots s = look(1);
    for (int j = 0; j < tiles; j += 2) {
      wait_lds();
      barrier();  // tile j is there, and the other pair is no longer read
      get_k(j + 1, k_b, s);
      get_v(j + 1, v_b, s);
      s = look(j + 2);
      score(j, k_a);
      weigh(j, v_a);
      if (j + 1 >= tiles) break;
      wait_lds();
      barrier();
      get_k(j + 2, k_a, s);
      get_v(j + 2, v_a, s);
      s = look(j + 3);
      score(j + 1, k_b);
      weigh(j + 1, v_b);
    }
  } else {
    // Phase p, one barrier each: waves 0 .. 3 score tile p / 2 in the even ones and
    // weigh it in the odd ones, waves 4 .. 7 one phase later. K of tile j + 1 is
    // copied from the end of phase 2 j (its place was last read in 2 j - 1) and
    // first read in 2 j + 2; V of tile j + 1 from the end of 2 j + 1 (last read in
    // 2 j) for 2 j + 3: each has a whole phase, and is waited for at its end.
    auto k_end = [&](int j, T *kt, const Spots &s) __attribute__((always_inline)) {
      wait_lds();
      get_k(j, kt, s);
      barrier();
    };
    auto v_end = [&](int j, T *vt, const Spots &s) __attribute__((always_inline)) {
      wait_lds();
      get_v(j, vt, s);
      barrier();
    };
    Spots s = look(1);
    wait_lds();
    barrier();
    if (w < 4) {
      for (int j = 0; j < tiles; j += 2) {
        score(j, k_a);
        k_end(j + 1, k_b, s);
        weigh(j, v_a);
        v_end(j + 1, v_b, s);
        if (j + 1 >= tiles) break;
        s = look(j + 2);
        score(j + 1, k_b);
        k_end(j + 2, k_a, s);
        weigh(j + 1, v_b);
        v_end(j + 2, v_a, s);
        s = look(j + 3);
      }
      barrier();
    } else {
      k_end(1, k_b, s);
      for (int j = 0; j < tiles; j += 2) {
        score(j, k_a);
        v_end(j + 1, v_b, s);
        s = look(j + 2);
        weigh(j, v_a);
        k_end(j + 2, k_a, s);
        if (j + 1 >= tiles) break;
        score(j + 1, k_b);
        v_end(j + 2, v_a, s);
        s = look(j + 3);
        weigh(j + 1, v_b);
        k_end(j + 3, k_b, s);
      }
    }
  }
  const int row = opaque<true>(32 * w + col);  // not kept along the loop
  const int token = t.q0 + row / share;
  x.store(row < tt * share && token < t.lq
              ? static_cast<T *>(a.o) +
                    ((int64_t)(t.qb + token) * a.h + t.group * share + row % share) * D
              : nullptr, hh);
}

// One part of a tile's keys, its running state left for a join. 128 rows: the more
// rows and parts, the more partial results are written and read again, so instead of
// taking 256 rows the eight waves are two sets of four, on the even and the odd tiles
// of the part, each with its own copies (double buffered). One barrier per step, the
// two waves of a SIMD overlap by chance: with a step of 32 keys (D = 256) the phases
// above cost more in barriers than they gain (39 against 36 us for 1024 rows on 8192
// keys of two heads). The second set's state is added to the first's through LDS at
// the end.
template <typename T, int D, Keys kKeys>
__global__ __launch_bounds__(512, 2) void attn_part_kernel(TileArgs a) {
  constexpr int kBM = 128, kBN = D == 256 ? 32 : 64;
  constexpr int kTile = kBN * D;
  // [set] [buffer] K and V; at the end, the second set's output sums
  __shared__ __attribute__((aligned(16))) T k_a[2 * kTile], v_a[2 * kTile], k_b[2 * kTile],
      v_b[2 * kTile];
  __shared__ float stat[4][64][2];
  __shared__ int scan[8][2];

  const int tid = threadIdx.x, lane = tid & 63, set = uniform(tid >> 8), w = uniform(tid >> 6) & 3;
  const int col = lane & 31, hh = lane >> 5;
  Where t;
  const int share = a.share, tt = kBM / share;
  if (!find<D, kKeys, true, 512>(a, tt, tid, t, scan)) return;
  t = t.uniform_();
  const int kvh = t.group * share / (a.h / a.hkv);
  const Sight see = sight_of<kKeys>(t, 32 * w, col, tt, share);
  const int all = see.keys > 0 ? (see.keys + kBN - 1) / kBN : 0;
  const int per = (all + a.splits - 1) / a.splits;
  const int j0 = t.split * per + set, end = min(t.split * per + per, all);
  const int steps = max((end - t.split * per + 1) / 2, 0);  // of either set
  // this set's tile of step j, if it has one
  auto has = [&](int j) { return j0 + 2 * j < end; };
  typedef Spot<Tile<T, D, kBN, 4>, kKeys> Spots;
  auto look = [&](int j) __attribute__((always_inline)) {
    Spots s = {};
    if (has(j)) s.look(a, t, (j0 + 2 * j) * kBN, w);
    return s;
  };
  Rows<T, D, kBN> x;
  auto walk = [&](auto past) __attribute__((always_inline)) {
    auto get_k = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
      if (has(j))
        get<T, D, kBN, 4, kKeys, false, decltype(past)::value>(a, t, s, kvh, (j0 + 2 * j) * kBN,
                                                               tile + set * kTile, lane, w);
    };
    auto get_v = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
      if (has(j))
        get<T, D, kBN, 4, kKeys, true, decltype(past)::value>(a, t, s, kvh, (j0 + 2 * j) * kBN,
                                                              tile + set * kTile, lane, w);
    };
    {
      const Spots s = look(0);
      get_k(0, k_a, s);
      get_v(0, v_a, s);
    }
    x.load(q_row<T>(a, t, see.tok, 32 * w + col, D), hh, a.scale_log2);
    auto score = [&](int j, T *kt) __attribute__((always_inline)) {
      const int k0 = (j0 + 2 * j) * kBN;
      if (has(j) && k0 <= see.hi)
        x.score((Lds<T>)(kt + set * kTile), k0, see.lim, k0 + kBN - 1 > see.lo, a.scale_log2, lane);
    };
    auto weigh = [&](int j, T *vt) __attribute__((always_inline)) {
      if (has(j) && (j0 + 2 * j) * kBN <= see.hi)
        x.weigh((Lds<T>)(vt + set * kTile), a.scale_log2, lane);
    };
    Spots s = look(1);
    for (int j = 0; j < steps; j += 2) {
      wait_lds();
      barrier();
      get_k(j + 1, k_b, s);
      get_v(j + 1, v_b, s);
      s = look(j + 2);
      score(j, k_a);
      weigh(j, v_a);
      if (j + 1 >= steps) break;
      wait_lds();
      barrier();
      get_k(j + 2, k_a, s);
      get_v(j + 2, v_a, s);
      s = look(j + 3);
      score(j + 1, k_b);
      weigh(j + 1, v_b);
    }
  };
  // (four contexts of 46000 tokens, 8 new ones each, 380 MB: 92 us, past the caches 87)
  if (kKeys == Keys::kPages && t.past_cache)
    walk(std::integral_constant<bool, kKeys == Keys::kPages>{});
  else
    walk(std::false_type{});
  wait_lds();
  barrier();  // the tiles are no longer read

  // the second set's state, lane by lane: a lane of both holds the same row and dims
  const Lds<T> tile = w == 0 ? (Lds<T>)k_a : w == 1 ? (Lds<T>)v_a : w == 2 ? (Lds<T>)k_b : (Lds<T>)v_b;
  const Lds<f32x4> mine = (Lds<f32x4>)tile;  // 32 rows of D floats
  if (set) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        mine[(4 * i + b) * 64 + lane] =
            f32x4{x.o[i][4 * b], x.o[i][4 * b + 1], x.o[i][4 * b + 2], x.o[i][4 * b + 3]};
    stat[w][lane][0] = x.m;
    stat[w][lane][1] = x.l;
  }
  __syncthreads();
  if (set) return;
  const float m2 = stat[w][lane][0], big = fmaxf(x.m, m2);
  const float f1 = x.m == kNegInf ? 0.f : fast_exp2(x.m - big);
  const float f2 = m2 == kNegInf ? 0.f : fast_exp2(m2 - big);
  x.m = big;
  x.l = x.l * f1 + stat[w][lane][1] * f2;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f32x4 y = mine[(4 * i + b) * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) x.o[i][4 * b + e] = x.o[i][4 * b + e] * f1 + y[e] * f2;
    }
  const int64_t at = (item_of(t.group, t.slot, a.h / share, a.slots) * a.splits + t.split) * kBM +
                     32 * w + col;
  x.store_part(a.part_o + at * D, a.part_ml + at * 2, hh);
}

// Joins the parts of a row's keys: one wave per row.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(TileArgs a, int tt, int bm) {
  constexpr int kPer = D / 64;  // dims per lane
  typedef float vec __attribute__((ext_vector_type(kPer)));
  const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
  const int64_t i = (int64_t)flat_block() * 4 + w;
  const int t = (int)(i / a.h), head = (int)(i % a.h);
  if (t >= cu_at(a.cu_q, a.n_max, a.t_max)) return;
  Tiled p;
  int first, total;
  auto none = [](int, int(&o)[2]) { o[0] = o[1] = 0; };
  auto in = [&](const auto &batch) {
    return batch.in_order(
        lane, [&](const Tiled &x, int, int) { return t >= x.b && t < x.b + x.n; }, p, first, total);
  };
  if (!(a.n_max <= 64 ? in(TiledBatch<1>(a.cu_q, a.n_max, a.t_max, tt, lane, none))
                      : in(TiledBatch<4>(a.cu_q, a.n_max, a.t_max, tt, lane, none))))
    return;  // an unsorted cu_seqlens: a row of no sequence
  const int tile = (t - p.b) / tt, slot = first + tile;
  if (slot >= a.slots) return;  // or sequences that overlap
  const int64_t item = item_of(head / a.share, slot, a.h / a.share, a.slots) * a.splits;
  const int row = (t - p.b - tile * tt) * a.share + head % a.share;
  // the splits' statistics, one per lane
  const float mine = lane < a.splits ? a.part_ml[((item + lane) * bm + row) * 2] : kNegInf;
  float big = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) big = fmaxf(big, __shfl_xor(big, off, 64));
  const float f = mine == kNegInf ? 0.f : fast_exp2(mine - big);
  float l = lane < a.splits ? a.part_ml[((item + lane) * bm + row) * 2 + 1] * f : 0.f;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) l += __shfl_xor(l, off, 64);
  vec sum = {};
  for (int k = 0; k < a.splits; k += 4) {  // four loads at a time
    vec x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = *reinterpret_cast<const vec *>(
          a.part_o + ((item + min(k + e, a.splits - 1)) * bm + row) * D + kPer * lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float g = __shfl(f, (k + e) & 63, 64);
      if (k + e < a.splits) sum += g * x[e];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<T *>(a.o) + ((int64_t)t * a.h + head) * D);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k)
    o[kPer / 2 * lane + k] = pack_mean<T>(sum[2 * k] * inv, sum[2 * k + 1] * inv);
}

template <typename T, int D, int kWaves, Keys kKeys>
hipError_t run_whole(const gdn_attn_config *cfg, const TileArgs &a, hipStream_t stream) {
  dim3 grid;
  if (!flat_grid((int64_t)a.slots * (cfg->h / a.share), 64 * kWaves, grid))
    return hipErrorInvalidValue;
  hipLaunchKernelGGL((attn_tile_kernel<T, D, kWaves, kKeys>), grid, dim3(64 * kWaves), 0, stream, a);
  return hipGetLastError();
}

template <typename T, int D, Keys kKeys>
hipError_t run_parts(const gdn_attn_config *cfg, const TileArgs &a, int tt, hipStream_t stream) {
  dim3 grid, join;
  if (!flat_grid((int64_t)a.slots * (cfg->h / a.share) * a.splits, 512, grid) ||
      !flat_grid(((int64_t)cfg->t_max * cfg->h + 3) / 4, 256, join))
    return hipErrorInvalidValue;
  hipLaunchKernelGGL((attn_part_kernel<T, D, kKeys>), grid, dim3(512), 0, stream, a);
  if (kKeys == Keys::kShared) return hipGetLastError();  // the caller joins them
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_tile_join_kernel<T, D>), join, dim3(256), 0, stream, a, tt, kPartRows);
  return hipGetLastError();
}

template <typename T, int D, Keys kKeys>
hipError_t run_keys(const gdn_attn_config *cfg, const TileArgs &a, const TileShape &s,
                    hipStream_t stream) {
  if (s.splits > 1) return run_parts<T, D, kKeys>(cfg, a, s.tt, stream);
  if constexpr (D == 256)
    return run_whole<T, D, 8, kKeys>(cfg, a, stream);
  else
    return s.waves == 8 ? run_whole<T, D, 8, kKeys>(cfg, a, stream)
                        : run_whole<T, D, 4, kKeys>(cfg, a, stream);
}

template <typename T, int D>
hipError_t run_of(const gdn_attn_config *cfg, Keys keys, const TileArgs &a, const TileShape &s,
                  hipStream_t stream) {
  return keys == Keys::kShared  ? run_parts<T, D, Keys::kShared>(cfg, a, s.tt, stream)
         : keys == Keys::kPages ? run_keys<T, D, Keys::kPages>(cfg, a, s, stream)
                                : run_keys<T, D, Keys::kRows>(cfg, a, s, stream);
}

// Average tokens per sequence from which heads of 128 take work-groups of eight
// waves: 4096 tokens 137 us against 140 us with four, 16384 tokens 955 against 968;
// 32 sequences of 500 on average 177 against 159 us.
constexpr int kLongPrompt = 2048;
// A tile's rows are tokens times the query heads that share a key head, as many
// of those as divide their number and are at most this many: tiles then span few
// tokens, so little is computed beyond the diagonal or past a sequence's end (32
// prompts of 500 tokens on average, two heads per key head: 176 -> 160 us).
constexpr int kMostShare = 16;
// A split has at least this many keys of the longest sequence that pages or the prefix can
// hold, or, of packed rows, of an average one, and there are at most 64 (one per lane of
// the join).
constexpr int kSplitKeys = 256;
constexpr int kMostSplits = 64;
// Tiles that fill the device between half and once are split in two: one prompt of 1200
// tokens with heads of 256 (150 tiles) 66 -> 50 us, of 2000 with heads of 128 (250) 58
// -> 50. A batch may be uneven and have more tiles than counted, so with several
// sequences only from this many keys on: 16 of 64 tokens on 2500 keys 140 -> 95 us; but
// 16 of 1 to 130 tokens on 1300 keys would go from 57 to 71, on 700 from 34 to 58.
constexpr int kTwoKeys = 2048;

}  // namespace

// Tiles of tt tokens have slots, t_max / tt + n_max at most; no table is needed to find
// a slot's tile. Up to kMostTiled sequences a wave counts the batch's tiles, the longest
// sequence's first (split: in order, the last first) and the slots left over last: where
// they lie between the tiles, a work-group without one costs a CU its turn (16
// sequences of 128 tokens on 2500 keys 165 us against 144, 64 of 32 on 1250: 130 against
// 96). Beyond, sequence s starts at slot floor(cu[s] / tt) + s, which is distinct for
// every tile of the batch and grows with s, and is found by a search.
TileShape tile_shape(const gdn_attn_config *cfg, Keys keys) {
  TileShape s;
  const int group = cfg->h / cfg->hkv;
  s.share = group < kMostShare ? group : kMostShare;
  while (group % s.share) --s.share;
  const int64_t room = (int64_t)cfg->max_pages * cfg->page_size;
  const int64_t longest = keys == Keys::kShared  ? (cfg->shared_max < room ? cfg->shared_max : room)
                          : keys == Keys::kPages ? room
                                                 : (cfg->tk_max > 0 ? cfg->tk_max : cfg->t_max) / cfg->n_max;
  auto cut = [&](int rows) {
    s.tt = rows / s.share;
    s.slots = keys == Keys::kShared ? (cfg->t_max + s.tt - 1) / s.tt : cfg->t_max / s.tt + cfg->n_max;
  };
  // few tiles (of a batch of equal sequences) and many keys: split the keys until the
  // device is full
  s.rows = kPartRows;
  s.waves = 8;
  cut(s.rows);
  const int64_t tiles =
      (keys == Keys::kShared ? s.slots
                             : (int64_t)cfg->n_max * ((cfg->t_max / cfg->n_max + s.tt - 1) / s.tt)) *
      (cfg->h / s.share);
  int64_t n = tiles > 0 ? cu_count() / tiles : 1;
  if (n == 1 && (cfg->n_max == 1 || longest >= kTwoKeys)) n = 2;
  if (n > longest / kSplitKeys) n = longest / kSplitKeys;
  s.splits = n < 1 ? 1 : n > kMostSplits ? kMostSplits : static_cast<int>(n);
  if (keys != Keys::kShared && cfg->n_max > kMostTiled) s.splits = 1;
  if (s.splits > 1 || keys == Keys::kShared) return s;
  s.waves = cfg->d == 256 || cfg->t_max / cfg->n_max >= kLongPrompt ? 8 : 4;
  s.rows = 32 * s.waves;
  cut(s.rows);
  return s;
}

int64_t tile_part_rows(const gdn_attn_config *cfg, const TileShape &s, Keys keys) {
  if (s.splits == 1 && keys != Keys::kShared) return 0;
  return (int64_t)s.slots * (cfg->h / s.share) * s.splits * s.rows;
}

hipError_t launch_attn_tiles(const gdn_attn_config *cfg, Keys keys, TileArgs a, hipStream_t stream) {
  if (cfg->t_max == 0) return hipSuccess;
  const TileShape s = tile_shape(cfg, keys);
  a.share = s.share;
  a.splits = s.splits;
  a.slots = s.slots;
  if (cfg->dtype == GDN_BF16)
    return cfg->d == 128 ? run_of<__bf16, 128>(cfg, keys, a, s, stream)
                         : run_of<__bf16, 256>(cfg, keys, a, s, stream);
  return cfg->d == 128 ? run_of<_Float16, 128>(cfg, keys, a, s, stream)
                       : run_of<_Float16, 256>(cfg, keys, a, s, stream);
}

}  // namespace gdn
