// Attention of a few new tokens per sequence to a paged cache (decode, verify).
//
// The rows of an item are the new tokens of one sequence times the query heads of one
// key / value head, 16 kRT at a time; an item's keys are cut into units of 128. Pages
// that the whole batch shares can come before: the part kernel of the tiles has then
// taken all rows past them and left partial results, and the items start behind them.
//
// HBM-bound on the keys and values, each read once per item: 256 sequences of about 2500
// keys (2.7 GB) 422 us, 6.4 TB/s, where a large copy reaches 5.0 and a large sum, which
// only reads, 4.0. Few keys are bound by latency: one token on 1000 keys 13 us, of which the
// main kernel 8.7. 128 tokens behind 8192 shared positions 70 us: the prefix 35, the
// sequences' own 250 keys 25, the join 9.
//
//  * Work: all units of the batch in one line (key head, sequences in order, row
//    tiles, units), cut into equal runs, one per work-group of a fixed grid. So
//    lengths need not be known on the host, a single long sequence fills the
//    device, and a ragged batch is balanced to one unit. A run covers the end of one
//    item, whole items, and the start of another. Whole items are written at once;
//    the others leave (maximum, sum, output sum) in the workspace, at most two per
//    work-group, and the join kernel adds them up, row by row.
//  * Each of the four waves takes 32 keys of a unit on its own, with a running
//    maximum and sum of its own; the waves meet once per item, in LDS. There is
//    no barrier in the loop over keys.
//  * K and V go from the pages to registers in 16-byte loads, in the layout of
//    the matrix instructions: scores S^T = K Q^T (a lane's column is one row),
//    O^T += V^T P^T. K's fragment is 8 consecutive dims of one key, as stored.
//    For V a lane loads 8 keys x 8 dims (each instruction four whole rows of
//    256 bytes) and transposes the block inside its registers, one byte permute
//    per pair of values; fragment j then has the dims 8 c + j. The keys of a
//    lane are the ones its scores hold, so weights never leave the lane.
//  * 8-bit pages: the registers hold codes, half as many, and a fragment is turned into
//    16-bit values where it is used, two by an instruction. V's block is 8 keys x D / 16
//    dims a lane, transposed as bytes before. The bytes halve and the vector unit's work
//    grows by the conversions: 256 sequences of about 2500 keys 242 us (5.5 TB/s; 16-bit
//    422), one token on 1000 keys 12.9, 128 tokens behind 8192 shared positions 66.
#include "attn_common.hpp"
#include "attn_launch.hpp"

#include <type_traits>

namespace gdn {

namespace {

constexpr int kUnit = 128;  // keys per unit: 32 per wave

// What the join is told of a row (token and query head): the first work-group with a
// part of it, how many there are (0: it sees no key; 1: finished by one), and its
// number in the item's rows. Written by the work-group in whose run the item begins.
struct RowPlan {
  int first, parts, in_item, unused;
};

// Rows (tokens times query heads) from which the join takes one wave per row and not
// four: 8192 rows with a few parts at most 358 us with the main kernel against 362, 256
// rows with 16 parts 21.8 against 20.5.
constexpr int kManyRows = 4096;

// a / b for a >= 0, b > 0: mostly both fit 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
__device__ __forceinline__ int64_t lane_of(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)x, lane);
  return (int64_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32 | lo;
}

__device__ __forceinline__ int units_of(int keys) { return (keys + kUnit - 1) / kUnit; }

// Keys and values that are read once, by the one row tile of each item's heads, are read
// past the caches where those could not hold them (kPastCache):
// 256 sequences of 2500 keys 471 -> 441 us, 128 of 1250 with two heads of 256 80 -> 75; but
// 32 of 2200 (240 MB) would take 58 -> 53 from HBM and 48 -> 52 where the last call left them
// in the cache, 64 of 190 (50 MB) 25 -> 29. A batch in which some item has several row tiles
// leaves its keys in the caches for the next of them (400 new tokens on 4000 keys beside 63
// sequences of 500: 109 us, past the caches 146).
template <bool kPast>
__device__ __forceinline__ u32x4 load16(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kPast ? 2 : 0);  // 2: not temporal
}
template <bool kPast>
__device__ __forceinline__ u32x2 load8(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, kPast ? 2 : 0);
}

template <int kRT>
__device__ __forceinline__ int row_tiles(int rows) {
  return (int)(((int64_t)rows + 16 * kRT - 1) / (16 * kRT));
}

// A wave's 32 keys of a unit: K fragments of two tiles of 16, and rows of V (keys 4 g
// + e of tile 0, then of tile 1).
template <typename T, int D, bool k8>
struct Keys32 {
  typename Elem<T>::vec8 k[2][D / 32];
  u32x4 v[D / 128][8];
};
// The same in codes of an 8-bit cache, with each tile's scales. A lane's 16 bytes of a key are
// the fragments of two steps (dims 64 j + 16 g .., eight each); its part of a row of V
// is D / 16 dims in a row, from D / 16 * c on.
template <typename T, int D>
struct Keys32<T, D, true> {
  u32x4 k[2][D / 64];
  uint32_t v[8][D / 64];
  uint32_t k_scale[2], v_scale[2];
};

// The 4 x 4 bytes of four words the other way round: word i of the result has byte i of
// each.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                           uint32_t (&out)[4]) {
  const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab2 = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd2 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  out[0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(cd2, ab2, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(cd2, ab2, 0x07060302u);
}

template <typename T, int D, int kRT, bool k8>
__global__ __launch_bounds__(256, kRT * D <= 256 ? 2 : 1) void attn_stream_kernel(StreamArgs a) {
  typedef typename Elem<T>::vec8 vec8;
  constexpr int kRows = 16 * kRT;
  constexpr int kDC = D / 128;   // 128-dim blocks
  constexpr int kPad = D + 4;    // floats per row of the meeting place
  __shared__ __attribute__((aligned(16))) T qs[kRows][D + 8];
  __shared__ __attribute__((aligned(16))) float os[4][16][kPad];
  __shared__ float wm[4][kRows], wl[4][kRows];
  __shared__ int64_t scan64[5];
  __shared__ int scan32[4][2], again[4], found;

  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  // consecutive runs on one XCD: its L2 then holds the rows that they share
  const int wg = (blockIdx.x & 7) * ((a.grid + 7) / 8) + (blockIdx.x >> 3);
  if (wg >= a.grid) return;

  // ---- the plan: shared prefix, units of every sequence
  PagedBatch pg = a.pg;
  int G = a.h / a.hkv;
  const int prefix = shared_prefix<256>(pg, tid, scan32).len;
  auto units_in = [&](int s) __attribute__((always_inline)) -> int64_t {
    const Seq q = seq_at(pg, s);
    return q.n > 0 && q.kv > prefix ? (int64_t)row_tiles<kRT>(q.n * G) * units_of(q.kv - prefix) : 0;
  };
  // up to 64 sequences: one per lane, every wave for itself and without a barrier (one
  // sequence 13.4 -> 12.9 us); more: a stretch of them per thread
  const bool few = pg.n_max <= 64;
  const int per = (pg.n_max + 255) / 256;
  const int s0 = min(few ? lane : tid * per, pg.n_max);
  const int s1 = min(s0 + (few ? 1 : per), pg.n_max);
  int64_t mine = 0;
  bool twice = false;  // keys that more than one row tile reads
  for (int s = s0; s < s1; ++s) {
    const int64_t u = units_in(s);
    mine += u;
    twice = twice || (u > 0 && row_tiles<kRT>(seq_at(pg, s).n * G) > 1);
  }
  twice = __any(twice);
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t y = __shfl_up(incl, off, 64);
    if (lane >= off) incl += y;
  }
  int64_t before = incl - mine, per_head;
  if (few) {
    per_head = lane_of(incl, 63);
  } else {
    if (lane == 63) scan64[w] = incl, again[w] = twice;
    __syncthreads();
    per_head = 0;
    for (int i = 0; i < 4; ++i) {
      if (i < w) before += scan64[i];
      per_head += scan64[i];
      twice = twice || again[i];
    }
    per_head = uniform(per_head);
  }
  const int64_t total = per_head * a.hkv;
  const int64_t per_wg = max(quotient(total + a.grid - 1, a.grid), (int64_t)1);
  const bool past = uniform(total > kPastCache / (kUnit * D * (k8 ? 2 : 4)) && !twice);
  RowPlan *const plan = reinterpret_cast<RowPlan *>(a.plan);
  if (wg == 0 && (!few || w == 0)) {
    if (tid == 0) a.prefix[0] = prefix, a.prefix[1] = past;
    // rows of sequences without keys belong to no item
    for (int s = s0; s < s1; ++s) {
      const Seq q = seq_at(pg, s);
      if (q.kv <= prefix)
        for (int64_t i = 0; i < (int64_t)q.n * a.h; ++i)
          plan[(int64_t)q.bos * a.h + i] = RowPlan{0, 0, 0, 0};
    }
  }
  const int64_t u0 = (int64_t)wg * per_wg, u1 = min(u0 + per_wg, total);
  if (u0 >= u1) return;

  // ---- the item of u0: the lane or thread whose sequences hold it names it
  int kh = (int)quotient(u0, per_head);
  int64_t in_head = u0 - kh * per_head;
  const bool here = in_head >= before && in_head < before + mine;
  int s;
  int64_t in_seq;
  if (few) {
    s = __ffsll((unsigned long long)__ballot(here)) - 1;
    in_seq = in_head - lane_of(before, s);
  } else {
    if (here) {
      int64_t at = before;
      int i = s0;
      for (int64_t n = units_in(i); in_head >= at + n; n = units_in(i)) {
        at += n;
        ++i;
      }
      found = i;
      scan64[4] = in_head - at;
    }
    __syncthreads();
    s = uniform(found);
    in_seq = uniform(scan64[4]);
  }
  // From here on everything but the lanes' data is one value per wave. The compiler
  // would merge what the branch above derived from these into lane values.
  G = uniform(G);
  pg.n_max = uniform(pg.n_max);
  pg.t_max = uniform(pg.t_max);
  pg.n_pages = uniform(pg.n_pages);
  pg.max_pages = uniform(pg.max_pages);
  pg.page_shift = uniform(pg.page_shift);

  typedef std::conditional_t<k8, uint8_t, T> Held;  // what the pages hold
  const Held *kpool = static_cast<const Held *>(a.k_pages), *vpool = static_cast<const Held *>(a.v_pages);
  auto walk = [&](auto past) __attribute__((always_inline)) {
    int64_t u = u0;
    while (u < u1) {
      // the item: its rows, its keys, the units of it in this run
      const int seq = uniform(s), head = uniform(kh);
      const Seq at = seq_at(pg, seq);
      const Seq q{uniform(at.bos), uniform(at.n), uniform(at.kv)};
      const int nu = units_of(q.kv - prefix);
      // (one value per wave each, which the compiler does not see by itself)
      const int rt = uniform((int)quotient(in_seq, nu)), un = uniform((int)(in_seq - (int64_t)rt * nu));
      const int run = uniform((int)min((int64_t)(nu - un), u1 - u));
      const int rows = q.n * G, r0 = rt * kRows;  // at most t_max * h, which fits

      // this wave's 32 keys of unit i of the run, as two tiles of 16, each in one page
      const int first = prefix + un * kUnit + 32 * w;
      const int mine_n = min(run, units_of(q.kv - first));  // units in which it has keys
      auto tile_key = [&](int i, int t) { return min(first + i * kUnit + 16 * t, (q.kv - 1) & ~15); };
      int pages[2];
      auto look = [&](int i) __attribute__((always_inline)) {
  #pragma unroll
        for (int t = 0; t < 2; ++t) pages[t] = page_of(pg, seq, tile_key(i, t));
      };
      // a tile's rows as a range that ends with the sequence's last key: zeros past it,
      // where a page may hold anything
      auto rows_of = [&](const Held *pool, int i, int t) __attribute__((always_inline)) {
        const int left = q.kv - (first + i * kUnit + 16 * t);
        const Held *p = pool + pool_row(pg, pages[t], tile_key(i, t), head, a.hkv) * D;
        return make_rsrc(p, uniform(max(min(left, 16), 0)) * D * (int)sizeof(Held));
      };
      typedef Keys32<T, D, k8> Unit;
      auto load_k = [&](Unit &x, int i) __attribute__((always_inline)) {
  #pragma unroll
        for (int t = 0; t < 2; ++t) {
          const rsrc_t r = rows_of(kpool, i, t);
          if constexpr (k8) {
            x.k_scale[t] = a.k_scales[scale_at(pg, pages[t], tile_key(i, t), head, a.hkv)];
  #pragma unroll
            for (int j = 0; j < D / 64; ++j)
              x.k[t][j] = load16<decltype(past)::value>(r, c * D + 16 * g + 64 * j);
          } else {
  #pragma unroll
            for (int j = 0; j < D / 32; ++j)
              x.k[t][j] = __builtin_bit_cast(
                  vec8, load16<decltype(past)::value>(r, (c * D + 8 * g + 32 * j) * 2));
          }
        }
      };
      auto load_v = [&](Unit &x, int i) __attribute__((always_inline)) {
  #pragma unroll
        for (int t = 0; t < 2; ++t) {
          const rsrc_t r = rows_of(vpool, i, t);
          if constexpr (k8) {
            x.v_scale[t] = a.v_scales[scale_at(pg, pages[t], tile_key(i, t), head, a.hkv)];
  #pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (D == 128) {
                const u32x2 y = load8<decltype(past)::value>(r, (4 * g + e) * D + 8 * c);
                x.v[4 * t + e][0] = y[0];
                x.v[4 * t + e][1] = y[1];
              } else {
                const u32x4 y = load16<decltype(past)::value>(r, (4 * g + e) * D + 16 * c);
  #pragma unroll
                for (int k = 0; k < 4; ++k) x.v[4 * t + e][k] = y[k];
              }
            }
          } else {
  #pragma unroll
            for (int e = 0; e < 4; ++e)
  #pragma unroll
              for (int b = 0; b < kDC; ++b)
                x.v[b][4 * t + e] =
                    load16<decltype(past)::value>(r, ((4 * g + e) * D + 128 * b + 8 * c) * 2);
          }
        }
      };
      Unit x;
      if (mine_n > 0) {
        look(0);
        load_k(x, 0);
        load_v(x, 0);
        if (mine_n > 1) look(1);
      }
      // the rows, while the first keys come
      __syncthreads();  // the item before may still be read
      for (int i = tid; i < kRows * (D / 8); i += 256) {
        const int row = i / (D / 8), ch = i % (D / 8);
        const int r = min(r0 + row, rows - 1), tok = r / G;
        *reinterpret_cast<u32x4 *>(&qs[row][8 * ch]) = *reinterpret_cast<const u32x4 *>(
            static_cast<const T *>(a.q) + (int64_t)(q.bos + tok) * a.q_row +
            (head * G + (r - tok * G)) * D + 8 * ch);
      }
      if (un == 0 && tid < kRows && r0 + tid < rows) {
        const int r = r0 + tid, tok = r / G;
        const int64_t over = u + nu - u1;  // units of the item past this run
        const int parts = over > 0 ? (int)quotient(over + per_wg - 1, per_wg) + 1 : 1;
        plan[(int64_t)(q.bos + tok) * a.h + head * G + (r - tok * G)] = RowPlan{wg, parts, tid, 0};
      }
      int lim[kRT];  // the last key that this lane's row of each tile sees
  #pragma unroll
      for (int t = 0; t < kRT; ++t) lim[t] = q.kv - q.n + min(r0 + 16 * t + c, rows - 1) / G;
      const int all_see = q.kv - q.n + r0 / G;  // every row sees these
      __syncthreads();

      f32x4 o[kRT][kDC][8];
      float m[kRT], l[kRT];
      int far[kRT];  // whether some row's maximum is past kFarLog2
  #pragma unroll
      for (int t = 0; t < kRT; ++t) {
        m[t] = kNegInf;
        l[t] = 0.f;
        far[t] = 0;
  #pragma unroll
        for (int b = 0; b < kDC; ++b)
  #pragma unroll
          for (int j = 0; j < 8; ++j) o[t][b][j] = zero4();
      }
      // the next keys come while these are weighed, the next values while their scores
      // are formed, in the registers that are free by then
      for (int i = 0; i < mine_n; ++i) {
        const int k0 = first + i * kUnit;
        const bool masked = k0 + 31 > all_see;
        // q's fragments are read anew for every unit (with one tile of 128 dims they fit
        // the registers and the compiler keeps them)
        const int qrow = opaque<(kRT * D > 128)>(c);
        f32x4 sc[kRT][2];
  #pragma unroll
        for (int t = 0; t < kRT; ++t) sc[t][0] = sc[t][1] = zero4();
        if constexpr (k8) {
          // (a fragment is formed once, for all row tiles)
          const T *const q0 = &qs[qrow][16 * g];
  #pragma unroll
          for (int p = 0; p < D / 32; ++p)
  #pragma unroll
            for (int k = 0; k < 2; ++k) {
              const vec8 kf = __builtin_bit_cast(
                  vec8, values8<T>(x.k[k][p >> 1][2 * (p & 1)], x.k[k][p >> 1][2 * (p & 1) + 1],
                                   scale_of(x.k_scale[k])));
  #pragma unroll
              for (int t = 0; t < kRT; ++t)
                sc[t][k] = mfma(kf, *reinterpret_cast<const vec8 *>(
                                        q0 + 16 * t * (D + 8) + 64 * (p >> 1) + 8 * (p & 1)),
                                sc[t][k]);
            }
        } else {
  #pragma unroll
          for (int t = 0; t < kRT; ++t)
  #pragma unroll
            for (int p = 0; p < D / 32; ++p) {
              const vec8 qf = *reinterpret_cast<const vec8 *>(&qs[16 * t + qrow][32 * p + 8 * g]);
              sc[t][0] = mfma(x.k[0][p], qf, sc[t][0]);
              sc[t][1] = mfma(x.k[1][p], qf, sc[t][1]);
            }
        }
        if (i + 1 < mine_n) load_k(x, i + 1);
        __builtin_amdgcn_sched_barrier(0);
        vec8 pf[kRT];
  #pragma unroll
        for (int t = 0; t < kRT; ++t) {
          if (masked) {
  #pragma unroll
            for (int e = 0; e < 8; ++e)
              if (k0 + 16 * (e >> 2) + 4 * g + (e & 3) > lim[t]) sc[t][e >> 2][e & 3] = kNegInf;
          }
          float mx = fmaxf(fmaxf(fmaxf(sc[t][0][0], sc[t][0][1]), fmaxf(sc[t][0][2], sc[t][0][3])),
                           fmaxf(fmaxf(sc[t][1][0], sc[t][1][1]), fmaxf(sc[t][1][2], sc[t][1][3])));
          mx = max32(max16(mx)) * a.scale_log2;
          if (__any(mx > m[t] + kRescaleLog2)) {
            const float mn = fmaxf(m[t], mx);
            const float al = mn == kNegInf ? 1.f : fast_exp2(m[t] - mn);
            m[t] = mn;
            l[t] *= al;
  #pragma unroll
            for (int b = 0; b < kDC; ++b)
  #pragma unroll
              for (int j = 0; j < 8; ++j) o[t][b][j] *= al;
            far[t] = __any(m[t] != kNegInf && fabsf(m[t]) > kFarLog2);
          }
          float ms = m[t] == kNegInf ? 0.f : m[t], scale = a.scale_log2;
          if (far[t]) {
  #pragma unroll
            for (int e = 0; e < 8; ++e)
              sc[t][e >> 2][e & 3] = far_exponent(sc[t][e >> 2][e & 3], scale, ms);
            ms = 0.f;
            scale = 1.f;
          }
          ms -= Elem<T>::kWeightLog2;
          u32x4 pw;
  #pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float e0 = fast_exp2(fmaf(sc[t][e >> 1][2 * (e & 1)], scale, -ms));
            const float e1 = fast_exp2(fmaf(sc[t][e >> 1][2 * (e & 1) + 1], scale, -ms));
            l[t] += e0 + e1;
            pw[e] = Elem<T>::pack(e0, e1);
          }
          pf[t] = __builtin_bit_cast(vec8, pw);
        }
        if constexpr (k8) {
          // four dims at a time: the bytes of a word, of the lane's eight keys
  #pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            uint32_t lo[4], hi[4];
            transpose4(x.v[0][k], x.v[1][k], x.v[2][k], x.v[3][k], lo);
            transpose4(x.v[4][k], x.v[5][k], x.v[6][k], x.v[7][k], hi);
  #pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float s0 = scale_of(x.v_scale[0]), s1 = scale_of(x.v_scale[1]);
              const vec8 vf = __builtin_bit_cast(
                  vec8, u32x4{values2<T, false>(lo[j], s0), values2<T, true>(lo[j], s0),
                              values2<T, false>(hi[j], s1), values2<T, true>(hi[j], s1)});
              const int b = k >> 1, at = 4 * (k & 1) + j;
  #pragma unroll
              for (int t = 0; t < kRT; ++t) o[t][b][at] = mfma(vf, pf[t], o[t][b][at]);
            }
          }
        } else
  #pragma unroll
        for (int b = 0; b < kDC; ++b)
  #pragma unroll
          for (int j = 0; j < 8; ++j) {
            u32x4 y;
  #pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = __builtin_amdgcn_perm(x.v[b][2 * e + 1][j >> 1], x.v[b][2 * e][j >> 1],
                                           j & 1 ? 0x07060302u : 0x05040100u);
            const vec8 vf = __builtin_bit_cast(vec8, y);
  #pragma unroll
            for (int t = 0; t < kRT; ++t) o[t][b][j] = mfma(vf, pf[t], o[t][b][j]);
          }
        __builtin_amdgcn_sched_barrier(0);
        if (i + 1 < mine_n) load_v(x, i + 1);
        if (i + 2 < mine_n) look(i + 2);
      }

      // ---- the four waves meet, one 16-row tile at a time
  #pragma unroll
      for (int t = 0; t < kRT; ++t) {
        l[t] = sum32(sum16x(l[t]));
        if (g == 0) {
          wm[w][16 * t + c] = m[t];
          wl[w][16 * t + c] = l[t];
        }
      }
      const bool from_start = un == 0, to_end = un + run == nu;
      const bool whole = from_start && to_end;
      // whole and alone: the output; whole beside a prefix: the row's place; else
      // this work-group's place 0 (the item began before it) or 1 (it goes on)
      const bool last = whole && prefix == 0;
      const int64_t place = (int64_t)wg * 2 + (from_start ? 1 : 0);
  #pragma unroll
      for (int t = 0; t < kRT; ++t) {
        __syncthreads();
        float big = kNegInf;
  #pragma unroll
        for (int i = 0; i < 4; ++i) big = fmaxf(big, wm[i][16 * t + c]);
        const float f = m[t] == kNegInf ? 0.f : fast_exp2(m[t] - big);
  #pragma unroll
        for (int b = 0; b < kDC; ++b)
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            // (codes: a lane's dims of V are D / 16 in a row)
            float *p = &os[w][c][k8 ? D / 4 * g + D / 16 * i + 8 * b : 128 * b + 32 * g + 8 * i];
            const auto &x = o[t][b];
            *reinterpret_cast<f32x4 *>(p) = f32x4{x[0][i] * f, x[1][i] * f, x[2][i] * f, x[3][i] * f};
            *reinterpret_cast<f32x4 *>(p + 4) =
                f32x4{x[4][i] * f, x[5][i] * f, x[6][i] * f, x[7][i] * f};
          }
        __syncthreads();
        // sixteen threads per row, 4 dims each at a time
        const int row = tid >> 4, q4 = 4 * (tid & 15);
        const int r = r0 + 16 * t + row;
        if (r < rows) {
          float mm = kNegInf, ll = 0.f;
  #pragma unroll
          for (int i = 0; i < 4; ++i) mm = fmaxf(mm, wm[i][16 * t + row]);
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float mi = wm[i][16 * t + row];
            ll += wl[i][16 * t + row] * (mi == kNegInf ? 0.f : fast_exp2(mi - mm));
          }
          const int tok = r / G;
          const int64_t orow = (int64_t)(q.bos + tok) * a.h + head * G + (r - tok * G);
          const float inv = ll == 0.f ? 0.f : 1.f / ll;
          float *po, *pm;
          if (whole) {
            po = a.done_o + orow * D;
            pm = a.done_ml + orow * 2;
          } else {
            po = a.part_o + (place * kRows + 16 * t + row) * D;
            pm = a.part_ml + (place * kRows + 16 * t + row) * 2;
          }
          if (!last && (tid & 15) == 0) {
            pm[0] = mm;
            pm[1] = ll;
          }
  #pragma unroll
          for (int b = 0; b < D / 64; ++b) {
            f32x4 sum = zero4();
  #pragma unroll
            for (int i = 0; i < 4; ++i)
              sum += *reinterpret_cast<const f32x4 *>(&os[i][row][64 * b + q4]);
            if (last)
              *reinterpret_cast<u32x2 *>(static_cast<T *>(a.o) + orow * D + 64 * b + q4) =
                  u32x2{pack_mean<T>(sum[0] * inv, sum[1] * inv),
                        pack_mean<T>(sum[2] * inv, sum[3] * inv)};
            else
              *reinterpret_cast<f32x4 *>(po + 64 * b + q4) = sum;
          }
        }
      }

      // ---- the next item
      u += run;
      in_seq += run;
      in_head += run;
      if (u >= u1) break;
      if (in_head == per_head) {
        ++kh;
        in_head = in_seq = 0;
        s = 0;
        while (uniform(units_in(s)) == 0) ++s;
      } else if (in_seq == uniform(units_in(s))) {
        in_seq = 0;
        ++s;
        while (uniform(units_in(s)) == 0) ++s;
      }
    }
  };
  if (past)
    walk(std::true_type{});
  else
    walk(std::false_type{});
}

// Joins what several work-groups, the shared prefix's included, left of a row, and
// writes zeros where a row sees no key. kWaves waves per row (token and query head),
// each on every kWaves-th part; rows that the main kernel finished are left alone.
// The parts' statistics are read first, a lane each, so that the output sums, which
// are most of the bytes, are read without waiting for anything.
template <typename T, int D, int kRT, int kWaves>
__global__ __launch_bounds__(256) void attn_stream_join_kernel(StreamArgs a) {
  constexpr int kRows = 16 * kRT;
  constexpr int kPer = D / 64;  // dims per lane
  typedef float vec __attribute__((ext_vector_type(kPer)));
  __shared__ float os[kWaves][64][kPer], stat[kWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int64_t row = (int64_t)flat_block() * (4 / kWaves) + (kWaves == 1 ? w : 0);
  const int t = (int)(row / a.h), head = (int)(row % a.h);
  const int sub = kWaves == 1 ? 0 : w;  // this wave among the row's
  if (t >= a.pg.t_max) return;
  const RowPlan plan = reinterpret_cast<const RowPlan *>(a.plan)[row];
  const int prefix = a.prefix[0];
  if (t >= cu_at(a.pg.cu, a.pg.n_max, a.pg.t_max)) return;
  // (an unsorted cu_seqlens leaves rows without a plan: whatever it holds is kept in range)
  const int w0 = min(max(uniform(plan.first), 0), a.grid - 1);
  const int parts = min(max(uniform(plan.parts), 0), a.grid - w0);
  const int in_item = uniform(plan.in_item) & (kRows - 1);
  const int lead = prefix > 0 ? a.pre_splits : 0;  // the prefix's parts come first
  if (lead == 0 && parts == 1) return;  // the main kernel wrote it
  const int64_t pre_item =
      (int64_t)(a.pre_slots - 1 - t / a.pre_tt) * (a.h / a.pre_share) + head / a.pre_share;
  const int pre_row = t % a.pre_tt * a.pre_share + head % a.pre_share;
  const int n = lead + parts;
  auto where = [&](int i, const float *&po, const float *&pm) __attribute__((always_inline)) {
    if (i < lead) {
      const int64_t at = (pre_item * a.pre_splits + i) * a.pre_rows + pre_row;
      po = a.pre_o + at * D;
      pm = a.pre_ml + at * 2;
    } else if (parts == 1) {
      po = a.done_o + row * D;
      pm = a.done_ml + row * 2;
    } else {
      // place 1 of the work-group in which the item begins, place 0 of the others
      const int64_t at = ((int64_t)(w0 + i - lead) * 2 + (i == lead ? 1 : 0)) * kRows + in_item;
      po = a.part_o + at * D;
      pm = a.part_ml + at * 2;
    }
  };
  // running state of this wave's parts: sub, sub + kWaves, ..., 64 at a time
  float big = kNegInf, l = 0.f;
  vec sum = {};
  for (int base = sub; base < n; base += 64 * kWaves) {
    const int mine = base + lane * kWaves, here = min(64, (n - base + kWaves - 1) / kWaves);
    const float *po, *pm;
    where(min(mine, n - 1), po, pm);
    const float m = mine < n ? pm[0] : kNegInf;
    float top = m;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    const float now = fmaxf(big, top);
    const float old = big == kNegInf ? 0.f : fast_exp2(big - now);
    const float f = m == kNegInf ? 0.f : fast_exp2(m - now);
    float add = pm[1] * f;  // (a sum that is NaN stays, also beside a maximum of -inf)
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) add += __shfl_xor(add, off, 64);
    big = now;
    l = l * old + add;
    sum *= old;
    for (int k = 0; k < here; k += 4) {  // four loads at a time
      vec x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        where(min(base + (k + e) * kWaves, n - 1), po, pm);
        x[e] = *reinterpret_cast<const vec *>(po + kPer * lane);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float g = __shfl(f, (k + e) & 63, 64);
        if (k + e < here) sum += g * x[e];
      }
    }
  }
  if constexpr (kWaves > 1) {
    *reinterpret_cast<vec *>(os[sub][lane]) = sum;
    if (lane == 0) stat[sub][0] = big, stat[sub][1] = l;
    __syncthreads();
    if (sub) return;
    const float mine = big;
    for (int i = 1; i < kWaves; ++i) big = fmaxf(big, stat[i][0]);
    const float f = mine == kNegInf ? 0.f : fast_exp2(mine - big);
    l *= f;
    sum *= f;
    for (int i = 1; i < kWaves; ++i) {
      const float g = stat[i][0] == kNegInf ? 0.f : fast_exp2(stat[i][0] - big);
      l += stat[i][1] * g;
      sum += *reinterpret_cast<const vec *>(os[i][lane]) * g;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<T *>(a.o) + row * D);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k)
    o[kPer / 2 * lane + k] = pack_mean<T>(sum[2 * k] * inv, sum[2 * k + 1] * inv);
}

template <typename T, int D, int kRT>
hipError_t run(const StreamArgs &a, int64_t rows, hipStream_t stream) {
  const bool wide = rows < kManyRows;
  dim3 join;
  if (!flat_grid(wide ? rows : (rows + 3) / 4, 256, join)) return hipErrorInvalidValue;
  const dim3 grid((a.grid + 7) / 8 * 8);
  if (a.k_scales)
    hipLaunchKernelGGL((attn_stream_kernel<T, D, kRT, true>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((attn_stream_kernel<T, D, kRT, false>), grid, dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (wide)
    hipLaunchKernelGGL((attn_stream_join_kernel<T, D, kRT, 4>), join, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((attn_stream_join_kernel<T, D, kRT, 1>), join, dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_of(const StreamArgs &a, int d, int rt, int64_t rows, hipStream_t stream) {
  if (d == 128)
    return rt == 1   ? run<T, 128, 1>(a, rows, stream)
           : rt == 2 ? run<T, 128, 2>(a, rows, stream)
                     : run<T, 128, 4>(a, rows, stream);
  return rt == 1 ? run<T, 256, 1>(a, rows, stream) : run<T, 256, 2>(a, rows, stream);
}

int64_t rows_per_seq(const gdn_attn_config *cfg) {
  return (int64_t)cfg->t_max * (cfg->h / cfg->hkv) / cfg->n_max;
}

}  // namespace

// Whether the prefix is worth a pass of its own: two launches more and a longer join
// (about 12 us) against reads of it by every sequence, of which most hit a cache. Even
// at 128 MiB of the latter (8 sequences on 16384 shared positions, 32 on 4096, 128 on
// 1024: 29 / 28 / 36 us against 30 / 25 / 29), ahead at 512 MiB (128 on 4096: 44
// against 57; with 4 times the heads and a quarter of the sequences 36 against 53). Over 8-bit
// pages by their own bytes: 128 MiB 44 against 33, 256 (128 sequences on 1024 positions, 32 on
// 4096, 8 on 16384) 48 / 35 / 33 against 57 / 53 / 54.
bool shares(const gdn_attn_config *cfg, bool k8) {
  constexpr double kWorth = 256.0 * (1 << 20);
  const double room = (double)cfg->max_pages * cfg->page_size;
  const double shared = cfg->shared_max < room ? cfg->shared_max : room;
  return shared * cfg->n_max * cfg->hkv * cfg->d * (k8 ? 2 : 4) >= kWorth;
}

// Rows of an average sequence (new tokens times query heads per key head) up to which
// its keys are streamed; with more, they are taken in tiles of 128 rows. With 32 rows
// both take as long (16 sequences on 2500 keys 44 us against 46, 64 on 1250: 91 against
// 86), with 64 the tiles are ahead (53 against 48, 116 against 90), except where only
// streamed items can leave the prefix to its own pass (64 sequences behind 8192 shared
// positions: 85 against 100; with 96 rows 124 against 102).
bool streams(const gdn_attn_config *cfg, bool k8) {
  return rows_per_seq(cfg) <= (shares(cfg, k8) ? 64 : 32);
}

// One 16-row tile per item holds a decoding sequence's heads; where an average
// sequence has more rows, wider items read the keys fewer times (32 rows on 2500 keys,
// 32 sequences: 84 us against 107; 64 rows: 107 against 199).
int stream_row_tiles(const gdn_attn_config *cfg) {
  const int most = cfg->d == 128 ? 4 : 2;
  int rt = 1;
  while (rt < most && rows_per_seq(cfg) > 16 * rt) rt *= 2;
  return rt;
}

int stream_grid(const gdn_attn_config *cfg) {
  return cu_count() * (stream_row_tiles(cfg) * cfg->d <= 256 ? 2 : 1);
}

hipError_t launch_attn_stream(const gdn_attn_config *cfg, StreamArgs a, hipStream_t stream) {
  if (cfg->t_max == 0) return hipSuccess;
  const int rt = stream_row_tiles(cfg);
  const int64_t rows = (int64_t)cfg->t_max * cfg->h;
  return cfg->dtype == GDN_BF16 ? run_of<__bf16>(a, cfg->d, rt, rows, stream)
                                : run_of<_Float16>(a, cfg->d, rt, rows, stream);
}

}  // namespace gdn
