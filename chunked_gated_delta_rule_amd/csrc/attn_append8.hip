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
// HBM-bound. A work-group takes the call's tokens of one block, 16 at most: so the block's
// scale is one wave's own, found in registers, without atomics and the same from run to
// run. Queries go row by row, as in the 16-bit front. A wave takes the 16 rows of one key
// head (64 / (D / 8) rows per step, a lane's eight channels of all of them in registers)
// or, with a single token, one row of several heads.
#include "attn_common.hpp"
#include "attn_launch.hpp"
#include "attn_row.hpp"

namespace gdn {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kBlock = 16;  // positions that share a scale

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

template <typename T, int D, Pairs kPairs, bool kAxes>
__global__ __launch_bounds__(kAppendThreads) void attn_append8_kernel(FrontArgs a) {
  constexpr int kLanes = D / 8;          // lanes per row
  constexpr int kStep = 64 / kLanes;     // rows of a wave at a time
  constexpr int kSteps = kBlock / kStep;
  __shared__ __attribute__((aligned(16))) float cs[kBlock][D / 2], sn[kBlock][D / 2];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int li = lane % kLanes, sub = lane / kLanes;
  const int half = a.rot_dim >> 1;
  const Channels<kPairs> ch(li, a.rot_dim);
  const int c0 = ch.c0, c1 = ch.c1;

  // ---- the block: block i of sequence s has slot floor(cu[s] / 16) + 2 s + i, distinct for
  // all (n tokens lie in (n + 30) / 16 blocks at most), and its tokens are lo .. hi - 1
  const int slot = flat_block();
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
  const int nt = hi - lo, t0 = p.b + lo;
  const int had = (int)max(pos0 - first, (int64_t)0);       // rows of the block before this call
  const T *const base = static_cast<const T *>(a.qkv) + (int64_t)t0 * a.qkv_row;

  // its place in a pool of one head, in rows, and its scale's in the scales of one head
  int64_t row0 = -1, at_scale = 0;
  const int per_page = 1 << (a.page_shift - 4);
  const int64_t col = first >> a.page_shift;
  if (first >= 0 && col < a.max_pages) {
    const int page = a.table[(int64_t)p.s * a.max_pages + col];
    if (page >= 0 && page < a.n_pages) {
      const int in = (int)(first & ((1 << a.page_shift) - 1));
      row0 = (((int64_t)page * a.hkv) << a.page_shift) + in;
      at_scale = ((int64_t)page * a.hkv) * per_page + in / kBlock;
    }
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
  typedef f32x4 weights __attribute__((aligned(4)));
  f32x4 wq0{1.f, 1.f, 1.f, 1.f}, wq1 = wq0, wk0 = wq0, wk1 = wq0;
  if (a.q_w) {
    wq0 = *reinterpret_cast<const weights *>(a.q_w + c0);
    wq1 = *reinterpret_cast<const weights *>(a.q_w + c1);
  }
  if (a.k_w) {
    wk0 = *reinterpret_cast<const weights *>(a.k_w + c0);
    wk1 = *reinterpret_cast<const weights *>(a.k_w + c1);
  }
  __syncthreads();

  // a row's values in fp32, of token tk and head hd (q, k and v in order)
  auto normed = [&](float(&x)[8], int tk, int hd, bool in) __attribute__((always_inline)) {
    const bool is_q = hd < a.h, is_v = hd >= a.h + a.hkv;
    if (is_v) return;
    norm_rope_row<T, D, kPairs>(
        x, ch, (is_q ? a.q_w : a.k_w) != nullptr, true, in, a.eps, a.rot_dim,
        [&](int j) __attribute__((always_inline)) {
          return j < 4 ? (is_q ? wq0[j & 3] : wk0[j & 3]) : (is_q ? wq1[j & 3] : wk1[j & 3]);
        },
        [&](const float *&ct, const float *&st) __attribute__((always_inline)) {
          ct = cs[tk];
          st = sn[tk];
        },
        [&]() __attribute__((always_inline)) { return base + tk * a.qkv_row + hd * D; },
        [&]() __attribute__((always_inline)) { return is_q ? a.q_w : a.k_w; });
  };
  auto store16 = [&](T *out, const float(&x)[8]) __attribute__((always_inline)) {
    *reinterpret_cast<u32x2 *>(out + c0) = u32x2{Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3])};
    *reinterpret_cast<u32x2 *>(out + c1) = u32x2{Elem<T>::pack(x[4], x[5]), Elem<T>::pack(x[6], x[7])};
  };

  // ---- keys and values: `heads` rows of heads side by side (a single token), or the rows
  // of one head
  auto keys = [&](auto single) __attribute__((always_inline)) {
    constexpr bool kOne = decltype(single)::value;
    constexpr int kR = kOne ? 1 : kSteps;
    const int items = kOne ? (2 * a.hkv + kStep - 1) / kStep : 2 * a.hkv;
    for (int item = w; item < items; item += kAppendThreads / 64) {
      const int kv = kOne ? item * kStep + sub : item;  // k of every head, then v
      const bool real = kv < 2 * a.hkv, is_v = kv >= a.hkv;
      const int kh = is_v ? kv - a.hkv : kv, hd = a.h + (real ? kv : 0);
      u32x2 y[kR][2];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int tk = kOne ? 0 : r * kStep + sub;
        y[r][0] = y[r][1] = u32x2{0u, 0u};
        if (tk < nt && real) {
          const T *row = base + tk * a.qkv_row + hd * D;
          y[r][0] = *reinterpret_cast<const u32x2 *>(row + c0);
          y[r][1] = *reinterpret_cast<const u32x2 *>(row + c1);
        }
      }
      uint8_t *const pool = static_cast<uint8_t *>(is_v ? a.v_pages : a.k_pages);
      uint8_t *const scales = is_v ? a.v_scales : a.k_scales;
      const bool placed = row0 >= 0 && real;
      const int64_t rows = row0 + ((int64_t)kh << a.page_shift);
      const int64_t my_scale = at_scale + (int64_t)kh * per_page;
      const int before = placed && had > 0 ? scales[my_scale] : 0;
      float x[kR][8], most = 0.f;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int tk = kOne ? 0 : r * kStep + sub;
        const bool in = tk < nt && real;
        unpack4<T>(y[r][0], x[r]);
        unpack4<T>(y[r][1], x[r] + 4);
        if (kOne || !is_v) {
          float z[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = x[r][j];
          normed(z, in ? tk : 0, is_v ? a.h : hd, in);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[r][j] = is_v ? x[r][j] : z[j];
          if (a.k && in && !is_v)
            store16(static_cast<T *>(a.k) + ((int64_t)(t0 + tk) * a.hkv + kh) * D, x[r]);
        }
        // what is not finite becomes NaN and does not count
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool finite = fabsf(x[r][j]) <= FLT_MAX;
          const float z = fminf(fmaxf(x[r][j], -kTop<T>), kTop<T>);
          if (in) most = fmaxf(most, finite ? fabsf(z) : 0.f);
          x[r][j] = finite ? z : __builtin_nanf("");
        }
      }
#pragma unroll
      for (int off = 1; off < (kOne ? kLanes : 64); off <<= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
      if (!placed) continue;
      const int e = max(scale_for(most), before);
      // the rows that the block had, by the new scale
      if (had > 0 && e > before) {
        const float by = __uint_as_float((uint32_t)max(before - e + 127, 1) << 23);
        for (int r = kOne ? 0 : sub; r < had; r += kOne ? 1 : kStep) {
          u32x2 *const at = reinterpret_cast<u32x2 *>(pool + (rows + r) * D + 8 * li);
          const u32x2 c = *at;
          *at = u32x2{again4(c[0], by), again4(c[1], by)};
        }
      }
      if (e != before && (kOne ? li == 0 : lane == 0)) scales[my_scale] = (uint8_t)e;
      const float by = unscale(e);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int tk = kOne ? 0 : r * kStep + sub;
        if (tk < nt) {
          uint8_t *const out = pool + (rows + had + tk) * D;
          const float *v = x[r];
          *reinterpret_cast<uint32_t *>(out + c0) = codes4(v[0] * by, v[1] * by, v[2] * by, v[3] * by);
          *reinterpret_cast<uint32_t *>(out + c1) = codes4(v[4] * by, v[5] * by, v[6] * by, v[7] * by);
        }
      }
    }
  };
  if (nt == 1)
    keys(std::true_type{});
  else
    keys(std::false_type{});

  // ---- queries, token by token, its heads in order
  if (!a.q) return;
  const int rows = nt * a.h;
  for (int at = 0; at < rows; at += kAppendThreads / kLanes) {
    const int r = at + tid / kLanes;
    const bool in = r < rows;
    const int tk = in ? r / a.h : 0, hd = in ? r - tk * a.h : 0;
    const T *row = base + tk * a.qkv_row + hd * D;
    float x[8];
    unpack4<T>(*reinterpret_cast<const u32x2 *>(row + c0), x);
    unpack4<T>(*reinterpret_cast<const u32x2 *>(row + c1), x + 4);
    normed(x, tk, hd, in);
    if (in) store16(static_cast<T *>(a.q) + ((int64_t)(t0 + tk) * a.h + hd) * D, x);
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
  dim3 grid;
  if (!flat_grid((int64_t)cfg->t_max / kBlock + 2 * (int64_t)cfg->n_max, kAppendThreads, grid))
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
