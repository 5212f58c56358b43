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
#include "attn_tile.hpp"

#include <type_traits>

namespace gdn {

namespace {

constexpr int kPartRows = 128;  // rows of a tile whose keys are split

// Whole tiles: kWaves waves of 32 rows. With four (D = 128, shorter sequences), three
// work-groups share a CU and overlap one's start and end with another's products; the
// keys go 32 at a time, for which the registers suffice (two work-groups and 64 keys:
// 128 sequences of 128 tokens 97 us against 85). With eight, the two waves of a SIMD (w
// and w + 4) go through the two parts of a step in opposite order, a barrier after each
// part: while one runs its score products the other forms weights (16384 tokens, 16
// heads of 256: 2658 us with four waves, 2130 with eight, when this was built; now 1900).
// Their steps have 64 keys, or 32 with heads of 256, which leaves registers to read
// fragments ahead (1836 -> 1820).
template <typename T, int D, int kWaves, Keys kKeys, bool k8>
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
  if (!find<kKeys, false, 64 * kWaves>(a, tt, D * (k8 ? 2 : 4), tid, t, scan)) return;
  t = t.uniform_();
  const int kvh = t.group * share / (a.h / a.hkv);
  const Sight see = sight_of<kKeys>(t, 32 * w, col, tt, share);
  const int tiles = see.keys > 0 ? (see.keys + kBN - 1) / kBN : 0;

  typedef Bring<T, D, kBN, kWaves, kKeys, k8> Brings;
  typedef typename Brings::Spots Spots;
  constexpr int kAhead = Brings::kAhead;
  Brings bring;
  auto look = [&](int j) __attribute__((always_inline)) {
    Spots s = {};
    if (k8 || j < tiles) s.look(a, t, j * kBN, w);
    return s;
  };
  auto key_of = [&](int j) { return j < tiles ? j * kBN : -1; };
  // tile j into LDS; s: the pages of tile j + kAhead
  auto get_k = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
    bring.template to<false, false>(tile, a, t, s, kvh, key_of(j), key_of(j + 1), lane, w);
  };
  auto get_v = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
    bring.template to<true, false>(tile, a, t, s, kvh, key_of(j), key_of(j + 1), lane, w);
  };
  Rows<T, D, kBN> x;
  {
    const Spots s = look(0);
    bring.template first<false, false>(a, t, s, kvh, key_of(0), lane, w);
    bring.template first<true, false>(a, t, s, kvh, key_of(0), lane, w);
    const Spots s1 = kAhead ? look(1) : s;
    get_k(0, k_a, s1);
    get_v(0, v_a, s1);
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
    Spots s = look(1 + kAhead);
    for (int j = 0; j < tiles; j += 2) {
      wait_tiles<k8>();
      barrier();  // tile j is there, and the other pair is no longer read
      get_k(j + 1, k_b, s);
      get_v(j + 1, v_b, s);
      s = look(j + 2 + kAhead);
      score(j, k_a);
      weigh(j, v_a);
      if (j + 1 >= tiles) break;
      wait_tiles<k8>();
      barrier();
      get_k(j + 2, k_a, s);
      get_v(j + 2, v_a, s);
      s = look(j + 3 + kAhead);
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
      wait_tiles<k8>();
      get_k(j, kt, s);
      barrier();
    };
    auto v_end = [&](int j, T *vt, const Spots &s) __attribute__((always_inline)) {
      wait_tiles<k8>();
      get_v(j, vt, s);
      barrier();
    };
    Spots s = look(1 + kAhead);
    wait_tiles<k8>();
    barrier();
    if (w < 4) {
      for (int j = 0; j < tiles; j += 2) {
        score(j, k_a);
        k_end(j + 1, k_b, s);
        weigh(j, v_a);
        v_end(j + 1, v_b, s);
        if (j + 1 >= tiles) break;
        s = look(j + 2 + kAhead);
        score(j + 1, k_b);
        k_end(j + 2, k_a, s);
        weigh(j + 1, v_b);
        v_end(j + 2, v_a, s);
        s = look(j + 3 + kAhead);
      }
      barrier();
    } else {
      k_end(1, k_b, s);
      for (int j = 0; j < tiles; j += 2) {
        score(j, k_a);
        v_end(j + 1, v_b, s);
        s = look(j + 2 + kAhead);
        weigh(j, v_a);
        k_end(j + 2, k_a, s);
        if (j + 1 >= tiles) break;
        score(j + 1, k_b);
        v_end(j + 2, v_a, s);
        s = look(j + 3 + kAhead);
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
template <typename T, int D, Keys kKeys, bool k8>
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
  // The wave's rows: 32 from 32 rg on. Over codes the second set has them the other way round:
  // waves w and w + 4 share a SIMD, and a tile that is half full then keeps all four busy (4
  // sequences of 8 tokens, 64 rows each, on 43000 keys 88 -> 83 us when this was built).
  const int rg = k8 && set ? 3 - w : w;
  Where t;
  const int share = a.share, tt = kBM / share;
  constexpr bool kByKeys = k8 && kKeys == Keys::kPages;
  if (!find<kKeys, true, 512, kByKeys>(a, tt, D * (k8 ? 2 : 4), tid, t, scan)) return;
  t = t.uniform_();
  const int kvh = t.group * share / (a.h / a.hkv);
  const Sight see = sight_of<kKeys>(t, 32 * rg, col, tt, share);
  const int all = see.keys > 0 ? (see.keys + kBN - 1) / kBN : 0;
  const int per = (all + t.splits - 1) / t.splits;
  const int j0 = t.split * per + set, end = min(t.split * per + per, all);
  const int steps = max((end - t.split * per + 1) / 2, 0);  // of either set
  // this set's tile of step j, if it has one
  auto has = [&](int j) { return j0 + 2 * j < end; };
  typedef Bring<T, D, kBN, 4, kKeys, k8> Brings;
  typedef typename Brings::Spots Spots;
  constexpr int kAhead = Brings::kAhead;
  auto look = [&](int j) __attribute__((always_inline)) {
    Spots s = {};
    if (k8 || has(j)) s.look(a, t, (j0 + 2 * j) * kBN, w);
    return s;
  };
  auto key_of = [&](int j) { return has(j) ? (j0 + 2 * j) * kBN : -1; };
  Rows<T, D, kBN> x;
  auto walk = [&](auto past) __attribute__((always_inline)) {
    constexpr bool kPast = decltype(past)::value;
    Brings bring;
    // tile j into LDS; s: the pages of tile j + kAhead
    auto get_k = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
      bring.template to<false, kPast>(tile + set * kTile, a, t, s, kvh, key_of(j), key_of(j + 1), lane, w);
    };
    auto get_v = [&](int j, T *tile, const Spots &s) __attribute__((always_inline)) {
      bring.template to<true, kPast>(tile + set * kTile, a, t, s, kvh, key_of(j), key_of(j + 1), lane, w);
    };
    {
      const Spots s = look(0);
      bring.template first<false, kPast>(a, t, s, kvh, key_of(0), lane, w);
      bring.template first<true, kPast>(a, t, s, kvh, key_of(0), lane, w);
      const Spots s1 = kAhead ? look(1) : s;
      get_k(0, k_a, s1);
      get_v(0, v_a, s1);
    }
    x.load(q_row<T>(a, t, see.tok, 32 * rg + col, D), hh, a.scale_log2);
    auto score = [&](int j, T *kt) __attribute__((always_inline)) {
      const int k0 = (j0 + 2 * j) * kBN;
      if (has(j) && k0 <= see.hi)
        x.score((Lds<T>)(kt + set * kTile), k0, see.lim, k0 + kBN - 1 > see.lo, a.scale_log2, lane);
    };
    auto weigh = [&](int j, T *vt) __attribute__((always_inline)) {
      if (has(j) && (j0 + 2 * j) * kBN <= see.hi)
        x.weigh((Lds<T>)(vt + set * kTile), a.scale_log2, lane);
    };
    Spots s = look(1 + kAhead);
    for (int j = 0; j < steps; j += 2) {
      wait_tiles<k8>();
      barrier();
      get_k(j + 1, k_b, s);
      get_v(j + 1, v_b, s);
      s = look(j + 2 + kAhead);
      score(j, k_a);
      weigh(j, v_a);
      if (j + 1 >= steps) break;
      wait_tiles<k8>();
      barrier();
      get_k(j + 2, k_a, s);
      get_v(j + 2, v_a, s);
      s = look(j + 3 + kAhead);
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
  const Lds<T> tile = rg == 0 ? (Lds<T>)k_a : rg == 1 ? (Lds<T>)v_a : rg == 2 ? (Lds<T>)k_b : (Lds<T>)v_b;
  const Lds<f32x4> mine = (Lds<f32x4>)tile;  // 32 rows of D floats
  if (set) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        mine[(4 * i + b) * 64 + lane] =
            f32x4{x.o[i][4 * b], x.o[i][4 * b + 1], x.o[i][4 * b + 2], x.o[i][4 * b + 3]};
    stat[rg][lane][0] = x.m;
    stat[rg][lane][1] = x.l;
  }
  __syncthreads();
  if (set) return;
  const float m2 = stat[rg][lane][0], big = fmaxf(x.m, m2);
  const float f1 = x.m == kNegInf ? 0.f : fast_exp2(x.m - big);
  const float f2 = m2 == kNegInf ? 0.f : fast_exp2(m2 - big);
  x.m = big;
  x.l = x.l * f1 + stat[rg][lane][1] * f2;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f32x4 y = mine[(4 * i + b) * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) x.o[i][4 * b + e] = x.o[i][4 * b + e] * f1 + y[e] * f2;
    }
  const int64_t item = kByKeys ? (int64_t)t.slot * (a.h / share) + t.group
                               : item_of(t.group, t.slot, a.h / share, a.slots) * a.splits + t.split;
  const int64_t at = item * kBM + 32 * rg + col;
  x.store_part(a.part_o + at * D, a.part_ml + at * 2, hh);
}

// Joins the parts of a row's keys: one wave per row.
template <typename T, int D, bool kByKeys>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(TileArgs a, int tt, int bm) {
  constexpr int kPer = D / 64;  // dims per lane
  typedef float vec __attribute__((ext_vector_type(kPer)));
  const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
  const int64_t i = (int64_t)flat_block() * 4 + w;
  const int t = (int)(i / a.h), head = (int)(i % a.h);
  if (t >= cu_at(a.cu_q, a.n_max, a.t_max)) return;
  // the row's parts: item(i) of the partial results, `splits` of them
  Tiled p;
  int splits, row;
  int64_t item, step;
  if constexpr (kByKeys) {
    int first;
    auto keys = [&](int i, int(&o)[2]) {
      o[0] = 0;
      o[1] = kv_of(a.pg, i);
    };
    auto in = [&](const auto &batch) {
      return batch.in_parts(
          lane, a.by_keys, kMostParts, kLeastKeys,
          [&](const Tiled &x, int, int) { return t >= x.b && t < x.b + x.n; }, p, first, splits);
    };
    if (!(a.n_max <= 64 ? in(TiledBatch<1>(a.cu_q, a.n_max, a.t_max, tt, lane, keys))
                        : in(TiledBatch<4>(a.cu_q, a.n_max, a.t_max, tt, lane, keys))))
      return;  // an unsorted cu_seqlens: a row of no sequence
    const int tile = (t - p.b) / tt;
    const int64_t at = first + (int64_t)tile * splits;
    if (at < 0 || at + splits > a.by_keys) return;  // or sequences that overlap
    step = a.h / a.share;
    item = at * step + head / a.share;
    row = (t - p.b - tile * tt) * a.share + head % a.share;
  } else {
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
    splits = a.splits;
    step = 1;
    item = item_of(head / a.share, slot, a.h / a.share, a.slots) * splits;
    row = (t - p.b - tile * tt) * a.share + head % a.share;
  }
  // the splits' statistics, one per lane
  const float mine = lane < splits ? a.part_ml[((item + lane * step) * bm + row) * 2] : kNegInf;
  float big = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) big = fmaxf(big, __shfl_xor(big, off, 64));
  const float f = mine == kNegInf ? 0.f : fast_exp2(mine - big);
  float l = lane < splits ? a.part_ml[((item + lane * step) * bm + row) * 2 + 1] * f : 0.f;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) l += __shfl_xor(l, off, 64);
  vec sum = {};
  for (int k = 0; k < splits; k += 4) {  // four loads at a time
    vec x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = *reinterpret_cast<const vec *>(
          a.part_o + ((item + min(k + e, splits - 1) * step) * bm + row) * D + kPer * lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float g = __shfl(f, (k + e) & 63, 64);
      if (k + e < splits) sum += g * x[e];
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
  if constexpr (kKeys != Keys::kRows) {
    if (a.k_scales) {
      hipLaunchKernelGGL((attn_tile_kernel<T, D, kWaves, kKeys, true>), grid, dim3(64 * kWaves), 0, stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((attn_tile_kernel<T, D, kWaves, kKeys, false>), grid, dim3(64 * kWaves), 0, stream, a);
  return hipGetLastError();
}

template <typename T, int D, Keys kKeys>
hipError_t run_parts(const gdn_attn_config *cfg, const TileArgs &a, int tt, hipStream_t stream) {
  dim3 grid, join;
  const int64_t parts = a.by_keys > 0 ? a.by_keys : (int64_t)a.slots * a.splits;
  if (!flat_grid(parts * (cfg->h / a.share), 512, grid) ||
      !flat_grid(((int64_t)cfg->t_max * cfg->h + 3) / 4, 256, join))
    return hipErrorInvalidValue;
  if constexpr (kKeys != Keys::kRows) {
    if (a.k_scales)
      hipLaunchKernelGGL((attn_part_kernel<T, D, kKeys, true>), grid, dim3(512), 0, stream, a);
    else
      hipLaunchKernelGGL((attn_part_kernel<T, D, kKeys, false>), grid, dim3(512), 0, stream, a);
  } else {
    hipLaunchKernelGGL((attn_part_kernel<T, D, kKeys, false>), grid, dim3(512), 0, stream, a);
  }
  if (kKeys == Keys::kShared) return hipGetLastError();  // the caller joins them
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if constexpr (kKeys == Keys::kPages) {
    if (a.by_keys > 0) {
      hipLaunchKernelGGL((attn_tile_join_kernel<T, D, true>), join, dim3(256), 0, stream, a, tt, kPartRows);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((attn_tile_join_kernel<T, D, false>), join, dim3(256), 0, stream, a, tt, kPartRows);
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
TileShape tile_shape(const gdn_attn_config *cfg, Keys keys, bool k8) {
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
  // Codes: the parts go by the sequences' keys, in as many work-groups as CUs, twice as many
  // where the tiles alone are more than half of that (us, equal parts against parts by keys:
  // 4 sequences of 8 tokens on 15000 to 60000 keys 61.6, 53.6; 16 of 16 on 1000 to 4000 35.6,
  // 33.8; 16 of 77 on 750 to 3000, heads of 256, 107, 104; one of 512 tokens on 8192 88.8,
  // 89.8. Twice the CUs throughout: 4 of 8 63, 16 of 16 43; once throughout: 16 of 77 124).
  s.by_keys = 0;
  if (k8 && keys == Keys::kPages && s.splits > 1) {
    const int64_t groups = cfg->h / s.share;
    const int64_t wgs = (tiles * 2 > cu_count() ? 2 : 1) * cu_count() / groups;
    s.by_keys = static_cast<int>(wgs > s.slots ? wgs : s.slots);
  }
  if (s.splits > 1 || keys == Keys::kShared) return s;
  s.waves = cfg->d == 256 || cfg->t_max / cfg->n_max >= kLongPrompt ? 8 : 4;
  s.rows = 32 * s.waves;
  cut(s.rows);
  return s;
}

int64_t tile_part_rows(const gdn_attn_config *cfg, const TileShape &s, Keys keys) {
  if (s.splits == 1 && keys != Keys::kShared) return 0;
  if (s.by_keys > 0) return (int64_t)s.by_keys * (cfg->h / s.share) * s.rows;
  return (int64_t)s.slots * (cfg->h / s.share) * s.splits * s.rows;
}

hipError_t launch_attn_tiles(const gdn_attn_config *cfg, Keys keys, TileArgs a, hipStream_t stream) {
  if (cfg->t_max == 0) return hipSuccess;
  const TileShape s = tile_shape(cfg, keys, a.k_scales != nullptr);
  a.share = s.share;
  a.splits = s.splits;
  a.slots = s.slots;
  a.by_keys = s.by_keys;
  if (cfg->dtype == GDN_BF16)
    return cfg->d == 128 ? run_of<__bf16, 128>(cfg, keys, a, s, stream)
                         : run_of<__bf16, 256>(cfg, keys, a, s, stream);
  return cfg->d == 128 ? run_of<_Float16, 128>(cfg, keys, a, s, stream)
                       : run_of<_Float16, 256>(cfg, keys, a, s, stream);
}

}  // namespace gdn
