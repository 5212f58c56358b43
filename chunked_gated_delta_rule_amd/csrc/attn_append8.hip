// Norm, rotation and the append to an 8-bit cache in one pass over the packed q | k | v rows.
//
// The cache holds e4m3 numbers and, for every 16 positions of a page and key head, the
// exponent byte e of a power of two: value = code * 2^(e - 127). A token's k (normed and
// turned, in fp32) or v is rounded once, to the code nearest to x * 2^(127 - e). With a = the
// largest |x| of the call's tokens in the block,
//
//   e = max(e before, the least e with a <= 448 * 2^(e - 127), 15)
//
// without `e before` where the block's first position is among the tokens. A power of two
// loses nothing to a scale with more digits, as the codes are floating-point numbers, and
// where a block's e grows, its rows by the new e are exact but for codes that get
// subnormal: they are read, rounded and written again by the wave that appends.
//
// HBM-bound where there are many tokens (32768 of 16 + 2 + 2 heads of 256: 133 us, 4.8 TB/s,
// where a large copy reaches 5.1; 2500 of 40 sequences, 32 + 4 + 4 heads of 128: 14.7, 3.3);
// one token for each of 256 sequences takes 7.6, the latency of finding the sequence, its
// page, the block's scale and rows, one after the other. A work-group takes the call's
// tokens of one block, 16 at most: so the block's scale is its own, found in registers and
// LDS, without atomics and the same from run to run.
// It goes through the heads in passes of 16 rows, D / 8 lanes and eight channels a lane, the
// next pass's loads in flight: first k and v, a pass having the rows of one head (of 16 /
// P heads, where P, the power of two that holds the tokens, is less than 16), then q
// token by token.
#include "attn_common.hpp"
#include "attn_launch.hpp"
#include "attn_row.hpp"

namespace gdn {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kBlock = 16;  // positions that share a scale
// Passes of a work-group where several share a block. What comes before the first pass is paid
// for by each, so as many as leave four work-groups per CU, within these limits (us with 2,
// 4, 6 and 8 throughout: 1024 tokens of 8 sequences, 16 + 2 + 2 heads of 256: 10.2, 13.4,
// 16.4, 19.2; 512 of one, 32 + 8 + 8 of 128: 7.4, 9.1, 11.2, 13.8; 2500 of 40 sequences 20.7,
// 16.9, 14.7, 15.3; 32768 of four 133, 133, 133, 141).
constexpr int kLeastPasses = 2, kMostPasses = 6;

// Largest finite value of the cache: the largest number of four significant bits that the
// 16-bit type holds, so that whoever reads the cache in that type finds no infinity.
template <typename T>
constexpr float kTop = 61440.f;
template <>
constexpr float kTop<__bf16> = 0x1.ep127f;

// The least scale: what is smaller than its steps vanishes (2^-121).
constexpr int kLeastScale = 15;

// e of the least power of two with a <= 448 * 2^(e - 127) (448 = 1.75 * 2^8), for finite a >= 0.
__device__ __forceinline__ int scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  return max((int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), kLeastScale);
}
// 2^(127 - e), for e in 1 .. 253.
__device__ __forceinline__ float unscale(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}
// Four codes times `by`, rounded again.
__device__ __forceinline__ uint32_t again4(uint32_t w, float by) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  return codes4(a[0] * by, a[1] * by, b[0] * by, b[1] * by);
}

// Maximum of the lanes of a row, in all of them (as sum16 and sum16x go).
template <int kLanes>
__device__ __forceinline__ float max_row(float x) {
  x = fmaxf(x, dpp_in<0xB1, 0xf>(x));
  x = fmaxf(x, dpp_in<0x4E, 0xf>(x));
  x = fmaxf(x, dpp_in<0x141, 0xf>(x));
  x = fmaxf(x, dpp_in<0x140, 0xf>(x));
  return kLanes == 32 ? max16(x) : x;
}

// A barrier for what is in LDS; loads go on coming (__syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <typename T, int D, Pairs kPairs, bool kAxes>
__global__ __launch_bounds__(kAppendThreads, 4) void attn_append8_kernel(FrontArgs a) {
  constexpr int kLanes = D / 8;                    // lanes per row
  constexpr int kRows = kAppendThreads / kLanes;   // rows at a time
  constexpr int kSub = kBlock / kRows;             // rows of a pass per thread: 1 or 2
  __shared__ __attribute__((aligned(16))) float cs[kBlock][D / 2], sn[kBlock][D / 2];
  __shared__ __attribute__((aligned(16))) float most[2][kBlock];
  const int tid = threadIdx.x, lane = tid & 63;
  const int li = tid % kLanes, at = tid / kLanes;
  const int half = a.rot_dim >> 1;
  const Channels<kPairs> ch(li, a.rot_dim);
  const int c0 = ch.c0, c1 = ch.c1;

  // ---- the block: block i of sequence s has slot floor(cu[s] / 16) + 2 s + i, distinct for
  // all (n tokens lie in (n + 30) / 16 blocks at most), and its tokens are lo .. hi - 1
  // (a.group blocks at a time, part by part. With groups of eight a block's parts are near in
  // time and all XCDs get as many of each; which part is first changes from group to group,
  // so that the shader engines do too)
  const int wg = flat_block(), group = wg / (a.group * a.parts), in = wg - group * a.group * a.parts;
  const int slot = a.group * group + in % a.group, part = (in / a.group + group) % a.parts;
  int lens[1];
  const Packed p = locate(
      a.cu, a.n_max, a.t_max, slot, lane, [](int s, int b) { return b / kBlock + 2 * s; },
      [&](int s, int(&o)[1]) { o[0] = a.kv_lens[s]; }, lens);
  const int i = slot - (p.b / kBlock + 2 * p.s);
  // (kv_lens is the caller's: positions are formed in 64 bits)
  const int64_t pos0 = (int64_t)lens[0] - p.n;              // of the sequence's first new token
  const int64_t first = ((pos0 >> 4) + i) * kBlock;         // of the block
  const int lo = (int)max(first - pos0, (int64_t)0);
  const int hi = (int)min(first + kBlock - pos0, (int64_t)p.n);
  if (i < 0 || lo >= hi) return;
  const int nt = uniform(hi - lo), t0 = uniform(p.b + lo);
  const int had = uniform((int)max(pos0 - first, (int64_t)0));  // rows of the block before this call
  const T *const base = static_cast<const T *>(a.qkv) + (int64_t)t0 * a.qkv_row;

  // ---- passes: kp of k and as many of v, P token slots per head, then q; this work-group's
  // share of them
  const int shift = nt > 1 ? 32 - __builtin_clz(nt - 1) : 0;  // P = 1 << shift
  const int kp = (a.hkv + (kBlock >> shift) - 1) >> (4 - shift), kvp = 2 * kp;
  const int all = kvp + (a.q ? (nt * a.h + kBlock - 1) / kBlock : 0);
  const int per = (all + a.parts - 1) / a.parts, pass0 = part * per, passes = min(pass0 + per, all);
  if (pass0 >= passes) return;
  // (offsets are in 32 bits: 16 rows of 2^24 values at most, heads of 256 in pages of 256)
  const int row_len = (int)a.qkv_row;
  u32x2 y[kSub][2];
  auto load = [&](int u, int tk, int head) __attribute__((always_inline)) {
    const uint32_t r = (uint32_t)(tk * row_len + head * D);
    y[u][0] = *reinterpret_cast<const u32x2 *>(base + (r + c0));
    y[u][1] = *reinterpret_cast<const u32x2 *>(base + (r + c1));
  };
  auto unpack = [&](int u, float(&x)[8]) __attribute__((always_inline)) {
    unpack4<T>(y[u][0], x);
    unpack4<T>(y[u][1], x + 4);
  };
  typedef f32x4 weights __attribute__((aligned(4)));
  f32x4 w0, w1;  // the weights of the lane's channels
  auto weigh = [&](const float *w) __attribute__((always_inline)) {
    w0 = w ? *reinterpret_cast<const weights *>(w + c0) : f32x4{1.f, 1.f, 1.f, 1.f};
    w1 = w ? *reinterpret_cast<const weights *>(w + c1) : f32x4{1.f, 1.f, 1.f, 1.f};
  };
  // the row of token tk and head `head` of the packed row, weights w
  auto normed = [&](float(&x)[8], const float *w, int tk, int head, bool in) __attribute__((always_inline)) {
    norm_rope_row<T, D, kPairs>(
        x, ch, w != nullptr, true, in, a.eps, a.rot_dim,
        [&](int j) __attribute__((always_inline)) { return j < 4 ? w0[j & 3] : w1[j & 3]; },
        [&](const float *&ct, const float *&st) __attribute__((always_inline)) {
          ct = cs[tk];
          st = sn[tk];
        },
        [&]() __attribute__((always_inline)) { return base + (uint32_t)(tk * row_len + head * D); },
        [&]() __attribute__((always_inline)) { return w; });
  };
  auto store = [&](T *out, uint32_t to, const float(&x)[8]) __attribute__((always_inline)) {
    const u32x2 z0{Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3])};
    const u32x2 z1{Elem<T>::pack(x[4], x[5]), Elem<T>::pack(x[6], x[7])};
    u32x2 *const p0 = reinterpret_cast<u32x2 *>(out + (to + c0)), *const p1 = reinterpret_cast<u32x2 *>(out + (to + c1));
    if (a.past_cache) {
      asm volatile("" ::: "memory");  // (the compiler would make one pair of the two)
      __builtin_nontemporal_store(z0, p0);
      __builtin_nontemporal_store(z1, p1);
      asm volatile("" ::: "memory");
    } else {
      *p0 = z0;
      *p1 = z1;
    }
  };

  // ---- keys and values. A slot without a token has its head all the same: it takes part
  // in what the head's block had
  auto kv_head = [&](int pass, int u) __attribute__((always_inline)) {
    return ((pass < kp ? pass : pass - kp) << (4 - shift)) + ((at + kRows * u) >> shift);
  };
  auto load_kv = [&](int pass) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      const int tk = (at + kRows * u) & ((1 << shift) - 1);
      load(u, tk < nt ? tk : 0, min(kv_head(pass, u), a.hkv - 1) + a.h + (pass < kp ? 0 : a.hkv));
    }
  };
  const int q0 = max(pass0 - kvp, 0), q_end = passes - kvp;  // passes of q
  int q_tok[kSub], q_head[kSub];
  auto load_q = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kSub; ++u) load(u, q_tok[u] < nt ? q_tok[u] : 0, q_tok[u] < nt ? q_head[u] : 0);
  };
  if (pass0 < kvp) {
    load_kv(pass0);
    weigh(a.k_w);
  } else {
    weigh(a.q_w);
  }
  if (q0 < q_end) {
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      const int r = q0 * kBlock + at + kRows * u;
      q_tok[u] = r / a.h;
      q_head[u] = r - q_tok[u] * a.h;
    }
    if (pass0 >= kvp) load_q();
  }

  for (int x = tid; x < nt * half; x += kAppendThreads) {
    const int k = x / half, j = x - k * half;
    double pos;
    if constexpr (kAxes)
      pos = a.positions[min(max(a.pair_axis[j], 0), a.n_axes - 1) * (int64_t)a.t_max + t0 + k];
    else
      pos = (double)(pos0 + lo + k);
    const f32x2 turn = turn_of(pos, a.inv_freq[j], a.rot_scale);
    cs[k][j] = turn[0];
    sn[k][j] = turn[1];
  }
  lds_barrier();

  if (pass0 < kvp) {
    // the block's place in a pool, in rows of head 0, and its scale's
    int64_t row0 = -1, at_scale = 0;
    const int page_size = 1 << a.page_shift, per_page = page_size / kBlock;
    const int64_t col = first >> a.page_shift;
    if (first >= 0 && col < a.max_pages) {
      const int page = a.table[(int64_t)p.s * a.max_pages + col];
      if (page >= 0 && page < a.n_pages) {
        const int in = (int)(first & (page_size - 1));
        row0 = (((int64_t)page * a.hkv) << a.page_shift) + in;
        at_scale = ((int64_t)page * a.hkv) * per_page + in / kBlock;
      }
    }
    row0 = uniform(row0);
    at_scale = uniform(at_scale);
    for (int pass = pass0; pass < min(passes, kvp); ++pass) {
      const bool is_v = pass >= kp;
      float x[kSub][8];
      int head[kSub], before[kSub];
      uint8_t *const scales = (is_v ? a.v_scales : a.k_scales) + at_scale;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        unpack(u, x[u]);
        head[u] = min(kv_head(pass, u), a.hkv - 1);
        before[u] = row0 >= 0 && had > 0 ? scales[(uint32_t)(head[u] * per_page)] : 0;
      }
      if (pass + 1 < min(passes, kvp))
        load_kv(pass + 1);
      else if (q0 < q_end)
        load_q();
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int slot_tk = (at + kRows * u) & ((1 << shift) - 1), tk = slot_tk < nt ? slot_tk : 0;
        const bool in = slot_tk < nt && kv_head(pass, u) < a.hkv;
        if (!is_v) {
          normed(x[u], a.k_w, tk, a.h + head[u], in);
          if (a.k && in)
            store(static_cast<T *>(a.k) + (int64_t)t0 * a.hkv * D, (uint32_t)((tk * a.hkv + head[u]) * D), x[u]);
        }
        // what is not finite becomes NaN and does not count
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool finite = fabsf(x[u][j]) <= FLT_MAX;
          const float v = fminf(fmaxf(x[u][j], -kTop<T>), kTop<T>);
          m = fmaxf(m, finite ? fabsf(v) : 0.f);
          x[u][j] = finite ? v : __builtin_nanf("");
        }
        m = max_row<kLanes>(m);
        if (li == 0) most[pass & 1][at + kRows * u] = in ? m : 0.f;
        // (here by now: after the barrier another wave of the head may write a new one)
        asm volatile("" : "+v"(before[u]));
      }
      lds_barrier();
      if (row0 < 0) continue;
      uint8_t *const pool = static_cast<uint8_t *>(is_v ? a.v_pages : a.k_pages) + row0 * D;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int s = at + kRows * u, tk = s & ((1 << shift) - 1);
        float m = 0.f;
        const float *of = &most[pass & 1][s - tk];
        for (int r = 0; r < 1 << shift; ++r) m = fmaxf(m, of[r]);
        const int e = max(scale_for(m), before[u]);
        if (kv_head(pass, u) >= a.hkv) continue;
        const uint32_t row = (uint32_t)(head[u] << a.page_shift);  // the head's first, from row0
        // the rows that the block had, by the new scale
        if (had > 0 && e > before[u]) {
          const float by = __uint_as_float((uint32_t)max(before[u] - e + 127, 1) << 23);
          for (int r = tk; r < had; r += 1 << shift) {
            u32x2 *const old = reinterpret_cast<u32x2 *>(pool + (row + r) * D + 8 * li);
            const u32x2 c = *old;
            *old = u32x2{again4(c[0], by), again4(c[1], by)};
          }
        }
        if (e != before[u] && tk == 0 && li == 0) scales[(uint32_t)(head[u] * per_page)] = (uint8_t)e;
        if (tk < nt) {
          const float by = unscale(e), *v = x[u];
          const uint32_t to = (row + had + tk) * D;
          *reinterpret_cast<uint32_t *>(pool + (to + c0)) = codes4(v[0] * by, v[1] * by, v[2] * by, v[3] * by);
          *reinterpret_cast<uint32_t *>(pool + (to + c1)) = codes4(v[4] * by, v[5] * by, v[6] * by, v[7] * by);
        }
      }
    }
    weigh(a.q_w);
  }

  // ---- queries, token by token, its heads in order
  T *const out = static_cast<T *>(a.q) + (int64_t)t0 * a.h * D;
  for (int pass = q0; pass < q_end; ++pass) {
    float x[kSub][8];
    int tok[kSub], head[kSub];
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      unpack(u, x[u]);
      tok[u] = q_tok[u];
      head[u] = q_head[u];
      q_head[u] += kBlock;
      while (q_head[u] >= a.h) {
        q_head[u] -= a.h;
        ++q_tok[u];
      }
    }
    if (pass + 1 < q_end) load_q();
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      const bool in = tok[u] < nt;
      const int tk = in ? tok[u] : 0;
      normed(x[u], a.q_w, tk, in ? head[u] : 0, in);
      if (in) store(out, (uint32_t)((tk * a.h + head[u]) * D), x[u]);
    }
  }
}

template <typename T, int D, bool kAxes>
void run(const FrontArgs &a, bool interleaved, dim3 grid, hipStream_t stream) {
  const dim3 block(kAppendThreads);
  if (interleaved)
    hipLaunchKernelGGL((attn_append8_kernel<T, D, Pairs::kInterleaved, kAxes>), grid, block, 0, stream, a);
  else if (a.rot_dim % 8 == 0)
    hipLaunchKernelGGL((attn_append8_kernel<T, D, Pairs::kHalf, kAxes>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((attn_append8_kernel<T, D, Pairs::kHalfOdd, kAxes>), grid, block, 0, stream, a);
}

template <typename T, int D>
void run_of(const FrontArgs &a, bool interleaved, dim3 grid, hipStream_t stream) {
  a.positions ? run<T, D, true>(a, interleaved, grid, stream)
              : run<T, D, false>(a, interleaved, grid, stream);
}

}  // namespace

hipError_t launch_attn_append8(const gdn_attn_config *cfg, FrontArgs a, hipStream_t stream) {
  if (cfg->t_max == 0) return hipSuccess;
  // a block is shared by several work-groups until there are many per CU (32768 tokens of 20
  // heads of 256 in one part 153 us, 2: 141, 3 to 5: 133; 2500 tokens of 40 heads of 128 in
  // one 33, in six 14.7)
  const int64_t each = (cfg->t_max + cfg->n_max - 1) / cfg->n_max;  // tokens of an average sequence
  const int64_t blocks = cfg->n_max * ((each + kBlock - 1) / kBlock);
  const int64_t passes = ((each < kBlock ? each : kBlock) * (cfg->h + 2 * cfg->hkv) + kBlock - 1) / kBlock;
  const int64_t share = blocks * passes / (4 * cu_count());
  const int64_t least = share < kLeastPasses ? kLeastPasses : share > kMostPasses ? kMostPasses : share;
  int64_t parts = 32 * cu_count() / blocks;
  if (parts > passes / least) parts = passes / least;
  a.parts = parts > 1 ? (int)parts : 1;
  // where all of them run at once, the parts with k and v, which take longer, come first (the
  // 2500 tokens 18 -> 16; the 32768 would go from 133 to 138)
  const int64_t slots = (cfg->t_max / kBlock + 2 * (int64_t)cfg->n_max + 7) / 8 * 8;
  a.group = slots * a.parts <= 16 * cu_count() ? (int)slots : 8;
  const int64_t heads = (a.q ? cfg->h : 0) + (a.k ? cfg->hkv : 0) + cfg->hkv;  // (codes: two in one)
  a.past_cache = heads * cfg->t_max * cfg->d * 2 > kPastCache;
  dim3 grid;
  if (!flat_grid(slots * a.parts, kAppendThreads, grid))
    return hipErrorInvalidValue;
  const bool interleaved = cfg->rot_interleaved != 0;
  if (cfg->dtype == GDN_BF16)
    cfg->d == 128 ? run_of<__bf16, 128>(a, interleaved, grid, stream)
                  : run_of<__bf16, 256>(a, interleaved, grid, stream);
  else
    cfg->d == 128 ? run_of<_Float16, 128>(a, interleaved, grid, stream)
                  : run_of<_Float16, 256>(a, interleaved, grid, stream);
  return hipGetLastError();
}

}  // namespace gdn
