// Device-side building blocks shared by the softmax-attention kernels: 16-bit
// element types, packing, cross-lane steps, and the search of a packed batch.
#pragma once

#include "attn_launch.hpp"
#include "gdn_common.hpp"

namespace gdn {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// The two 16-bit element types: the MFMA operand vector, the rounding of a
// pair (to nearest even), and the value of the low and high half of a word.
// kWeightLog2: softmax weights, and with them their sum, are formed 2^kWeightLog2 times
// larger. fp16 has few exponents below 1: weights from 2^-21 of the row's largest on are
// then normal numbers, and smaller ones off by 2^-32 of it at most (2^-14 and 2^-25
// without). The largest can be 2^kRescaleLog2 times that, which fp16 still holds.
template <typename T>
struct Elem;
template <>
struct Elem<__bf16> {
  typedef bf16x8 vec8;
  static constexpr float kWeightLog2 = 0.f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
};
template <>
struct Elem<_Float16> {
  typedef f16x8 vec8;
  static constexpr float kWeightLog2 = 7.f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_f16(a, b); }
  static __device__ __forceinline__ float lo(uint32_t w) {
    return static_cast<float>(__builtin_bit_cast(f16x2, w)[0]);
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return static_cast<float>(__builtin_bit_cast(f16x2, w)[1]);
  }
};

// An output is a mean of values. The weights' roundings can take it past fp16's largest
// value, by 2^-11 of that at most, where a mean of finite values is not: the largest then.
constexpr float kPastF16 = 65520.f;  // from here on fp16 rounds to infinity
__device__ __forceinline__ float mean_f16(float x) {
  return fabsf(x) < 65600.f ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
}
template <typename T>
__device__ __forceinline__ uint32_t pack_mean(float a, float b) {
  if constexpr (__is_same(T, _Float16)) return Elem<T>::pack(mean_f16(a), mean_f16(b));
  return Elem<T>::pack(a, b);
}

// Maximum and sum over lanes l and l ^ 32 (l ^ 16), in both: the swap of half
// (quarter) waves leaves the lower ones' values in one register and the upper
// ones' in the other.
struct Halves {
  float a, b;
};
__device__ __forceinline__ Halves halves32(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Halves halves16(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ float max32(float x) {
  const Halves h = halves32(x);
  return fmaxf(h.a, h.b);
}
__device__ __forceinline__ float sum32(float x) {
  const Halves h = halves32(x);
  return h.a + h.b;
}
__device__ __forceinline__ float max16(float x) {
  const Halves h = halves16(x);
  return fmaxf(h.a, h.b);
}
__device__ __forceinline__ float sum16x(float x) {
  const Halves h = halves16(x);
  return h.a + h.b;
}

// A value the compiler may not see through: what is derived from it is formed
// anew at each use, where keeping it would cost registers all along the loop.
template <bool kDo>
__device__ __forceinline__ int opaque(int x) {
  if constexpr (kDo) asm volatile("" : "+v"(x));
  return x;
}

constexpr float kNegInf = -__builtin_inff();

// Bytes from which what a pass reads or writes once goes past the caches: what the last
// level holds.
constexpr int64_t kPastCache = 256 << 20;

// Softmax statistics move only when a row's maximum (log2 scale) has grown by
// more than this: the weights then stay below 2^8 (fp16, formed larger: 2^15), in the
// range of 16 bits and of the fp32 sums, and the output sums are rescaled a few times
// per row only.
constexpr float kRescaleLog2 = 8.f;

// A weight's exponent, score * scale - m, is one fused step, so it contains the rounding of
// m = max * scale, up to 2^-24 |m|: a factor common to the row, which cancels. Past a maximum
// of this size the factor could leave the 16-bit types (past 2^32, fp32 as well: keys held
// off with the type's lowest value). The score and the maximum are then rounded alike
// before they are subtracted, which leaves 0 for equal ones.
constexpr float kFarLog2 = 1 << 20;
__device__ __forceinline__ float far_exponent(float score, float scale_log2, float m) {
  float s = score * scale_log2;
  asm("" : "+v"(s));  // (the two would be fused after all)
  return s - m;
}

// Narrows [0, n) to at most 64 indexes that hold the last s with key(s) <= x, for
// a non-decreasing key with key(0) <= x, by one wave: 64 probes per level (n <=
// 16384: at most two levels). [lo, lo + len) stays inside [0, n) for any key.
template <typename F>
__device__ __forceinline__ void narrow(int n, int x, int lane, int &lo, int &len, F key) {
  lo = 0;
  len = n;
  while (len > 64) {
    const int step = (len + 63) / 64;
    const int at = lane * step;
    const bool in = at < len && key(lo + at) <= x;
    const int skip = max((int)__popcll(__ballot(in)) - 1, 0) * step;
    lo += skip;
    len = min(step, len - skip);
  }
}

// A packed sequence: index, first row, rows.
struct Packed {
  int s, b, n;
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x);
  return (int64_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 | lo;
}

// The last sequence s of the batch whose key(s, first row of s) is at most x. Each
// lane of the last level loads what belongs to its sequence, extra(s) included,
// and the chosen lane's values are handed out: one round trip to memory for up to
// 64 sequences.
template <int kExtra, typename F, typename G>
__device__ __forceinline__ Packed locate(const int32_t *__restrict__ cu, int n_max, int t_max, int x,
                                         int lane, F key, G extra, int (&out)[kExtra]) {
  int lo, len;
  narrow(n_max, x, lane, lo, len, [&](int s) { return key(s, cu_at(cu, s, t_max)); });
  const int s = min(lo + lane, n_max - 1);
  const int b = cu_at(cu, s, t_max), n = cu_end(cu, s, b, t_max) - b;
  int mine[kExtra];
  extra(s, mine);
  const int hit = max((int)__popcll(__ballot(lane < len && key(s, b) <= x)) - 1, 0);
#pragma unroll
  for (int i = 0; i < kExtra; ++i) out[i] = __builtin_amdgcn_readlane(mine[i], hit);
  return {uniform(lo + hit), __builtin_amdgcn_readlane(b, hit), __builtin_amdgcn_readlane(n, hit)};
}

// Sequence of packed row t (t < cu[n_max]) and its value of `extra`.
template <typename G>
__device__ __forceinline__ Packed seq_of_row(const int32_t *__restrict__ cu, int n_max, int t_max,
                                             int t, int lane, G extra, int &out) {
  int v[1];
  const Packed p = locate(
      cu, n_max, t_max, t, lane, [](int, int b) { return b; },
      [&](int s, int(&o)[1]) { o[0] = extra(s); }, v);
  out = v[0];
  return p;
}

// A sequence of a batch of at most kMostTiled: index, first row, rows, and what extra(s)
// gave; its rows are cut into tiles of tt tokens.
struct Tiled {
  int s, b, n, extra[2];
};
constexpr int kMostTiled = 256;

// The batch in a wave, kPer (1 or 4) neighbouring sequences a lane, for n_max <= 64 kPer;
// all loads in one round trip. Sequences past n_max have no rows.
template <int kPer>
struct TiledBatch {
  Tiled seq[kPer];
  int tiles[kPer];

  template <typename G>
  __device__ __forceinline__ TiledBatch(const int32_t *__restrict__ cu, int n_max, int t_max, int tt,
                                        int lane, G extra) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      Tiled &p = seq[j];
      p.s = min(lane * kPer + j, n_max - 1);
      p.b = cu_at(cu, p.s, t_max);
      p.n = cu_end(cu, p.s, p.b, t_max) - p.b;
      extra(p.s, p.extra);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (lane * kPer + j >= n_max) seq[j].n = 0;
      tiles[j] = (seq[j].n + tt - 1) / tt;
    }
  }
  // The sequence for which a lane has found[j], in all lanes (false: none has; the
  // lowest lane's if several have, which an unsorted cu_seqlens can cause).
  __device__ __forceinline__ bool pick(const bool (&found)[kPer], Tiled &out) const {
    int v[5] = {seq[0].s, seq[0].b, seq[0].n, seq[0].extra[0], seq[0].extra[1]};
    bool any = found[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) {
      const bool take = found[j] && !any;
      v[0] = take ? seq[j].s : v[0];
      v[1] = take ? seq[j].b : v[1];
      v[2] = take ? seq[j].n : v[2];
      v[3] = take ? seq[j].extra[0] : v[3];
      v[4] = take ? seq[j].extra[1] : v[4];
      any = any || found[j];
    }
    const unsigned long long who = __ballot(any);
    if (who == 0) return false;
    const int hit = __ffsll(who) - 1;
    auto of = [&](int x) { return __builtin_amdgcn_readlane(x, hit); };
    out.s = of(v[0]);
    out.b = of(v[1]);
    out.n = of(v[2]);
    out.extra[0] = of(v[3]);
    out.extra[1] = of(v[4]);
    return true;
  }
  // Tiles numbered sequence by sequence without gaps: chosen(sequence, its first tile,
  // tiles of the batch) names one sequence; at and total are its values.
  template <typename F>
  __device__ __forceinline__ bool in_order(int lane, F chosen, Tiled &out, int &at, int &total) const {
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) mine += tiles[j];
    int end = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(end, off, 64);
      if (lane >= off) end += y;
    }
    total = __builtin_amdgcn_readlane(end, 63);
    int first = end - mine, which = 0;
    bool found[kPer], any = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      found[j] = !any && seq[j].n > 0 && chosen(seq[j], first, total);
      if (found[j]) which = first;
      any = any || found[j];
      first += tiles[j];
    }
    if (!pick(found, out)) return false;
    at = __builtin_amdgcn_readlane(which, __ffsll(__ballot(any)) - 1);
    return true;
  }
  // f over the wave's values: rows of 16 lanes (shifts by 1, 2, 4, 8), then the rows.
  template <typename F>
  static __device__ __forceinline__ int all(int v, F f) {
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true));
    return f(f(__builtin_amdgcn_readlane(v, 15), __builtin_amdgcn_readlane(v, 31)),
             f(__builtin_amdgcn_readlane(v, 47), __builtin_amdgcn_readlane(v, 63)));
  }
  // Tiles of the sequences that have at least x.
  __device__ __forceinline__ int from(int x) const {
    int v = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v += tiles[j] >= x ? tiles[j] : 0;
    return all(v, [](int a, int b) { return a + b; });
  }
  // Whether every sequence has one tile at most and the keys that extra[1] counts, of
  // `bytes` each, are more than the caches hold.
  __device__ __forceinline__ bool past_cache(int bytes) const {
    int v = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v += tiles[j] > 0 ? seq[j].extra[1] >> 8 : 0;
    const int64_t keys = (int64_t)all(v, [](int a, int b) { return a + b; }) << 8;
    return from(2) == 0 && keys * bytes > kPastCache;
  }
  // Tile number r with the longest sequence first and the last tile of each first:
  // tile is its index in the sequence. False: there are fewer tiles.
  __device__ __forceinline__ bool longest_first(int lane, int r, Tiled &out, int &tile) const {
    int most = tiles[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) most = max(most, tiles[j]);
    most = all(most, [](int a, int b) { return max(a, b); });
    // the sequence has x tiles: the largest x with more than r tiles in sequences that
    // have at least x
    int x = 0, before = 0;
    for (int bit = 1 << (31 - __builtin_clz(most | 1)); bit > 0; bit >>= 1) {
      const int c = from(x | bit);
      if (c > r)
        x |= bit;
      else
        before = c;  // (once all bits are tried: the tiles of sequences with more than x)
    }
    if (x == 0) return false;
    const int in = r - before, which = in / x;
    tile = x - 1 - (in - which * x);
    bool found[kPer];
    int seen = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const unsigned long long equal = __ballot(tiles[j] == x);
      const int rank = seen + (int)__popcll(equal & ((1ull << lane) - 1));
      found[j] = tiles[j] == x && rank == which;
      seen += (int)__popcll(equal);
    }
    return pick(found, out);
  }
};

// New tokens and keys of sequence s of a paged batch.
struct Seq {
  int bos, n, kv;
};
__device__ __forceinline__ int kv_of(const PagedBatch &a, int s) {
  const int64_t room = (int64_t)a.max_pages << a.page_shift;  // positions the table reaches
  const int kv = max(a.kv_lens[s], 0);
  return kv < room ? kv : (int)room;
}
__device__ __forceinline__ Seq seq_at(const PagedBatch &a, int s) {
  Seq q;
  q.bos = cu_at(a.cu, s, a.t_max);
  q.n = cu_end(a.cu, s, q.bos, a.t_max) - q.bos;
  q.kv = kv_of(a, s);
  return q;
}

// Page of position `key` of sequence s, as an index into the pool whatever the table
// says. s and key are uniform: the table is read through the scalar cache (which a
// plain load, next to stores, would not be).
__device__ __forceinline__ int page_of(const PagedBatch &a, int s, int key) {
  typedef __attribute__((address_space(4))) const int32_t *scalar;
  const scalar row = (scalar)(uintptr_t)(a.table + (int64_t)s * a.max_pages);
  return min(max(row[key >> a.page_shift], 0), a.n_pages - 1);
}
// Row of the pool at which position `key` of a key head lies in its page.
__device__ __forceinline__ int64_t pool_row(const PagedBatch &a, int page, int key, int kh, int hkv) {
  return (((int64_t)page * hkv + kh) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
}

// The shared prefix as it is used: whole pages, before every new token of the
// batch; and a sequence with new tokens, whose table leads to it. For a
// work-group of kThreads; `at` is its LDS.
struct Prefix {
  int len, seq;
};
template <int kThreads>
__device__ __forceinline__ Prefix shared_prefix(const PagedBatch &a, int tid,
                                                int (&at)[kThreads / 64][2]) {
  if (!a.shared_len || a.shared_max <= 0) return {0, 0};
  int least = min(max(a.shared_len[0], 0), a.shared_max), first = a.n_max;
  for (int s = tid; s < a.n_max; s += kThreads) {
    const Seq q = seq_at(a, s);
    if (q.n > 0) {
      least = min(least, q.kv - q.n);
      first = min(first, s);
    }
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    least = min(least, __shfl_xor(least, off, 64));
    first = min(first, __shfl_xor(first, off, 64));
  }
  if (tid % 64 == 0) at[tid / 64][0] = least, at[tid / 64][1] = first;
  __syncthreads();
  for (int i = 0; i < kThreads / 64; ++i) {
    least = min(least, at[i][0]);
    first = min(first, at[i][1]);
  }
  least = uniform(least);
  first = uniform(first);
  return {first < a.n_max ? max(least, 0) >> a.page_shift << a.page_shift : 0, min(first, a.n_max - 1)};
}

}  // namespace gdn
