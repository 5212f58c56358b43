// Front of a softmax-attention layer: RMS norm of every query and key head,
// rotation by the token's position, and (gdn_kv_append) the write of k and v
// into the pages of the cache, in one pass over the packed q | k | v rows.
//
//   x' = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> s (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[i]
//
// HBM-bound: each row is read once and written once (8192 tokens of 40 heads of 128: 36
// us, 4.6 TB/s, and 32 where the last-level cache still holds the rows; 32768 tokens of 20
// heads of 256 into pages: 127 us, 5.3 TB/s; a large copy reaches 5.0). 512 or fewer
// tokens take 6 us, most of it latency. A 256-thread work-group takes one or two
// tokens; D / 8 lanes own a head's row, eight channels each, and the work-group walks
// the heads of its tokens 2048 / D at a time, the next rows' loads in flight.
// The channels of a lane are chosen so that both members of its pairs are its own
// (half layout: four channels and the four rot_dim / 2 further; interleaved: eight in
// a row), so the rotation needs no other lane. Sequence, position, cache row, and the
// cos and sin of the rot_dim / 2 angles of each token are found once per work-group,
// in LDS, while the first rows' loads are in flight.
#include "attn_common.hpp"
#include "attn_launch.hpp"

#include <cfloat>
#include <type_traits>

namespace gdn {

namespace {

constexpr int kFrontThreads = 256;
// Tokens per work-group at most (32768 tokens of 20 heads of 256 from HBM 132 us, 8192 of
// 48 of 128 into pages 44; with one 142 and 43, four 136 and 49).
constexpr int kMostTokens = 2;

// How a lane's eight channels are placed: pairs inside the lane (half layout
// with rot_dim a multiple of 8, or interleaved), or (half layout with any other
// rot_dim) eight channels in a row whose partners are read one by one.
enum class Pairs { kHalf = 0, kInterleaved = 1, kHalfOdd = 2 };

// The least sum of squares that is taken as it is, and the factors for values whose sum is
// not fp32's (bf16 only): 2^128 2^-96 and 2^-126 2^96 have squares that are.
constexpr float kSmall = 0x1p-100f, kDown = 0x1p-96f, kUp = 0x1p96f;

// 1 / (2 pi), for angles counted in turns.
constexpr double kInvTwoPi = 0.15915494309189533577;

template <typename T>
__device__ __forceinline__ void unpack4(const u32x2 &w, float *f) {
  f[0] = Elem<T>::lo(w[0]);
  f[1] = Elem<T>::hi(w[0]);
  f[2] = Elem<T>::lo(w[1]);
  f[3] = Elem<T>::hi(w[1]);
}

// At least six waves per SIMD: the odd layout would take 82 registers, which leaves five (8192
// tokens of 40 heads of 128, rot_dim 34: 64 us against 58).
template <typename T, int D, Pairs kPairs, bool kCache>
__global__ __launch_bounds__(kFrontThreads, 6) void attn_front_kernel(FrontArgs a) {
  constexpr int kLanes = D / 8;                    // lanes per head
  constexpr int kRows = kFrontThreads / kLanes;    // rows per pass
  __shared__ __attribute__((aligned(16))) float cs[kMostTokens][D / 2], sn[kMostTokens][D / 2];
  __shared__ int64_t pos_of[kMostTokens], slot_of[kMostTokens];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int li = tid % kLanes;
  const int64_t t0 = (int64_t)flat_block() * a.tokens;
  const int half = a.rot_dim >> 1;

  // this lane's channels: c0 .. c0 + 3 and c1 .. c1 + 3
  int c0 = 8 * li, c1 = c0 + 4;
  bool turned = c0 < a.rot_dim;
  if constexpr (kPairs == Pairs::kHalf) {
    turned = li < half / 4;
    c0 = turned ? 4 * li : a.rot_dim + 8 * (li - half / 4);
    c1 = turned ? half + 4 * li : c0 + 4;
  }
  // rows of the work-group: token by token, its heads in order. The first ones are
  // asked for before it is known how many tokens there are (qkv has t_max rows)
  const int first = a.q ? 0 : a.h;
  const int heads = a.h + (kCache ? 2 : 1) * a.hkv - first;
  int rows = (int)min((int64_t)a.tokens, a.t_max - t0) * heads;
  const T *base = static_cast<const T *>(a.qkv) + t0 * a.qkv_row;
  int r = tid / kLanes, tok = r / heads, head = first + r - tok * heads;
  u32x2 x0{0u, 0u}, x1{0u, 0u};
  auto load = [&]() __attribute__((always_inline)) {
    if (r < rows) {
      const T *p = base + tok * a.qkv_row + head * D;
      x0 = *reinterpret_cast<const u32x2 *>(p + c0);
      x1 = *reinterpret_cast<const u32x2 *>(p + c1);
    }
  };
  load();
  const float freq = tid < half ? a.inv_freq[tid] : 0.f;
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
  const int total = cu_at(a.cu, a.n_max, a.t_max);
  if (t0 >= total) return;
  const int nt = min(a.tokens, total - (int)t0);
  rows = nt * heads;

  // (a single token: every wave for itself, and no barrier)
  for (int i = a.tokens > 1 ? w : 0; i < nt; i += kFrontThreads / 64) {
    const int t = (int)t0 + i;
    int len = 0;
    const Packed p = seq_of_row(
        a.cu, a.n_max, a.t_max, t, lane, [&](int s) { return a.kv_lens ? a.kv_lens[s] : 0; }, len);
    // kv_lens is the caller's: the position is formed in 64 bits
    const int64_t pos = a.kv_lens ? (int64_t)len - (p.b + p.n - t) : t - p.b;
    int64_t slot = -1;  // the token's row in a page pool of one head
    if constexpr (kCache) {
      const int64_t col = pos >> a.page_shift;
      if (pos >= 0 && col < a.max_pages) {
        const int page = a.table[(int64_t)p.s * a.max_pages + col];
        if (page >= 0 && page < a.n_pages)
          slot = (((int64_t)page * a.hkv) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
      }
    }
    if (lane == 0) {
      pos_of[i] = pos;
      slot_of[i] = slot;
    }
  }
  if (a.tokens > 1) __syncthreads();
  for (int i = tid; i < nt * half; i += kFrontThreads) {
    const int k = i / half, j = i - k * half;
    const float per_pos = k == 0 ? freq : a.inv_freq[j];
    const double turns = (double)pos_of[k] * (double)per_pos * kInvTwoPi;
    const float f = (float)(turns - __builtin_rint(turns));  // -1/2 .. 1/2
    cs[k][j] = a.rot_scale * __builtin_amdgcn_cosf(f);  // cos(2 pi f)
    sn[k][j] = a.rot_scale * __builtin_amdgcn_sinf(f);
  }
  __syncthreads();

  for (int at = 0; at < rows; at += kRows) {
    const bool in = r < rows;
    const u32x2 y0 = x0, y1 = x1;
    const int hd = head, tk = in ? tok : 0;
    r += kRows;
    head += kRows;
    while (head >= first + heads) {
      head -= heads;
      ++tok;
    }
    load();
    const bool is_q = hd < a.h, is_v = hd >= a.h + a.hkv;
    const bool norm = (is_q ? a.q_w : a.k_w) != nullptr && !is_v;
    float x[8];
    unpack4<T>(y0, x);
    unpack4<T>(y1, x + 4);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    ss = sum16(ss);
    if constexpr (kLanes == 32) ss = sum16x(ss);
    float rn = norm ? 1.f / sqrtf(ss * (1.f / D) + a.eps) : 1.f;
    float by = 1.f;
    if constexpr (std::is_same_v<T, __bf16>) {
      // values whose squares leave fp32 (past about 2^60), or vanish in it with nothing
      // added to them, are brought to the middle of its range first
      const bool large = ss > FLT_MAX, small = ss < kSmall && a.eps < kSmall;
      if (__any(norm && (large || small))) {
        if (norm && (large || small)) by = large ? kDown : kUp;
        ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] *= by;
          ss = fmaf(x[j], x[j], ss);
        }
        ss = sum16(ss);
        if constexpr (kLanes == 32) ss = sum16x(ss);
        if (norm) rn = 1.f / sqrtf(ss * (1.f / D) + a.eps * by * by);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] *= rn * (is_q ? wq0[j] : wk0[j]);
      x[j + 4] *= rn * (is_q ? wq1[j] : wk1[j]);
    }
    if (!is_v) {
      const float *ct = cs[tk], *st = sn[tk];
      if constexpr (kPairs == Pairs::kHalf) {
        if (turned) {
          const f32x4 c = *reinterpret_cast<const f32x4 *>(ct + c0);
          const f32x4 d = *reinterpret_cast<const f32x4 *>(st + c0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = x[j], v = x[j + 4];
            x[j] = u * c[j] - v * d[j];
            x[j + 4] = v * c[j] + u * d[j];
          }
        }
      } else if constexpr (kPairs == Pairs::kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (c0 + 2 * j < a.rot_dim) {
            const float c = ct[(c0 >> 1) + j], d = st[(c0 >> 1) + j];
            const float u = x[2 * j], v = x[2 * j + 1];
            x[2 * j] = u * c - v * d;
            x[2 * j + 1] = v * c + u * d;
          }
        }
      } else {
        if (in) {
          const float *wp = is_q ? a.q_w : a.k_w;
          const T *row = base + tk * a.qkv_row + hd * D;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = c0 + j;
            if (c < a.rot_dim) {
              const bool low = c < half;
              const int p = low ? c + half : c - half, i = low ? c : p;
              const float y = static_cast<float>(row[p]) * by * rn * (wp ? wp[p] : 1.f);
              x[j] = x[j] * ct[i] + (low ? -y : y) * st[i];
            }
          }
        }
      }
    }
    if (!in) continue;
    // v is copied as it is, bit for bit
    const u32x2 z0 = is_v ? y0 : u32x2{Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3])};
    const u32x2 z1 = is_v ? y1 : u32x2{Elem<T>::pack(x[4], x[5]), Elem<T>::pack(x[6], x[7])};
    auto store = [&](T *p) __attribute__((always_inline)) {
      u32x2 *const p0 = reinterpret_cast<u32x2 *>(p + c0), *const p1 = reinterpret_cast<u32x2 *>(p + c1);
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
    const int64_t t = t0 + tk;
    if (is_q) {
      store(static_cast<T *>(a.q) + (t * a.h + hd) * D);
      continue;
    }
    const int kh = hd - a.h - (is_v ? a.hkv : 0);
    if (!is_v && a.k) store(static_cast<T *>(a.k) + (t * a.hkv + kh) * D);
    if constexpr (kCache) {
      const int64_t slot = slot_of[tk];
      if (slot >= 0)
        store(static_cast<T *>(is_v ? a.v_pages : a.k_pages) +
              (slot + ((int64_t)kh << a.page_shift)) * D);
    }
  }
}

template <typename T, int D, bool kCache>
void run(const FrontArgs &a, bool interleaved, dim3 grid, hipStream_t stream) {
  const dim3 block(kFrontThreads);
  if (interleaved)
    hipLaunchKernelGGL((attn_front_kernel<T, D, Pairs::kInterleaved, kCache>), grid, block, 0,
                       stream, a);
  else if (a.rot_dim % 8 == 0)
    hipLaunchKernelGGL((attn_front_kernel<T, D, Pairs::kHalf, kCache>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((attn_front_kernel<T, D, Pairs::kHalfOdd, kCache>), grid, block, 0, stream,
                       a);
}

template <typename T>
void run_of(const FrontArgs &a, int d, bool interleaved, dim3 grid, hipStream_t stream) {
  if (d == 128)
    a.k_pages ? run<T, 128, true>(a, interleaved, grid, stream)
              : run<T, 128, false>(a, interleaved, grid, stream);
  else
    a.k_pages ? run<T, 256, true>(a, interleaved, grid, stream)
              : run<T, 256, false>(a, interleaved, grid, stream);
}

}  // namespace

hipError_t launch_attn_front(const gdn_attn_config *cfg, FrontArgs a, hipStream_t stream) {
  if (cfg->t_max == 0) return hipSuccess;
  // several tokens per work-group once there are enough for every CU's eight
  const int most = cfg->t_max / (8 * cu_count());
  a.tokens = most < 1 ? 1 : most > kMostTokens ? kMostTokens : most;
  // outputs that the caches could not hold for their reader are stored past them: 132 ->
  // 129 us at 335 MB, and with the attention that follows 16 prompts of 2048 tokens 722 ->
  // 715; 16 of 512 (84 MB) would go from 106 to 111
  const int64_t heads = (a.q ? cfg->h : 0) + (a.k ? cfg->hkv : 0) + (a.k_pages ? 2 * cfg->hkv : 0);
  a.past_cache = heads * cfg->t_max * cfg->d * 2 > kPastCache;
  dim3 grid;
  if (!flat_grid((cfg->t_max + a.tokens - 1) / a.tokens, kFrontThreads, grid))
    return hipErrorInvalidValue;
  if (cfg->dtype == GDN_BF16)
    run_of<__bf16>(a, cfg->d, cfg->rot_interleaved != 0, grid, stream);
  else
    run_of<_Float16>(a, cfg->d, cfg->rot_interleaved != 0, grid, stream);
  return hipGetLastError();
}

}  // namespace gdn
