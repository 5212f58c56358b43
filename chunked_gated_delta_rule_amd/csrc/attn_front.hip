// Front of a softmax-attention layer: RMS norm of every query and key head,
// rotation by the token's position (or, of a position of several axes, by the one that
// turns the pair), and (gdn_kv_append) the write of k and v into the pages of the cache,
// in one pass over the packed q | k | v rows.
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
#include "attn_row.hpp"

namespace gdn {

namespace {

constexpr int kFrontThreads = 256;
// Tokens per work-group at most (32768 tokens of 20 heads of 256 from HBM 132 us, 8192 of
// 48 of 128 into pages 44; with one 142 and 43, four 136 and 49).
constexpr int kMostTokens = 2;

// At least six waves per SIMD: the odd layout would take 82 registers, which leaves five (8192
// tokens of 40 heads of 128, rot_dim 34, from HBM: 86 us against 79).
//
// kAxes: positions of several axes come with the tokens, one axis for each pair of channels.
// They and the pairs' axes are asked for with the first rows, and without a cache no sequence
// is searched for: 8192 tokens of 40 heads of 128 35 us (4.8 TB/s), 512 of 18 of 256 5.9, as
// with one position per token; 24000 of 24 of 128 into pages 64 (4.7 TB/s).
template <typename T, int D, Pairs kPairs, bool kCache, bool kAxes>
__global__ __launch_bounds__(kFrontThreads, 6) void attn_front_kernel(FrontArgs a) {
  constexpr int kLanes = D / 8;                    // lanes per head
  constexpr int kRows = kFrontThreads / kLanes;    // rows per pass
  __shared__ __attribute__((aligned(16))) float cs[kMostTokens][D / 2], sn[kMostTokens][D / 2];
  __shared__ int64_t pos_of[kMostTokens], slot_of[kMostTokens];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t t0 = (int64_t)flat_block() * a.tokens;
  const int half = a.rot_dim >> 1;

  const Channels<kPairs> ch(tid % kLanes, a.rot_dim);
  const int c0 = ch.c0, c1 = ch.c1;
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
  int place = 0;  // where the token of this thread's first angle lies along the pair's axis
  if constexpr (kAxes) {
    static_assert(kMostTokens * (D / 2) <= kFrontThreads, "one angle per thread");
    const int k = half > 0 ? tid / half : 0, j = tid - k * half;
    if (half > 0 && k < a.tokens && t0 + k < a.t_max)
      place = a.positions[min(max(a.pair_axis[j], 0), a.n_axes - 1) * (int64_t)a.t_max + t0 + k];
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
  const int total = cu_at(a.cu, a.n_max, a.t_max);
  if (t0 >= total) return;
  const int nt = min(a.tokens, total - (int)t0);
  rows = nt * heads;

  // (a single token: every wave for itself, and no barrier)
  if constexpr (kCache || !kAxes) {
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
  }
  if (a.tokens > 1) __syncthreads();
  for (int i = tid; i < nt * half; i += kFrontThreads) {
    const int k = i / half, j = i - k * half;
    const float per_pos = k == 0 ? freq : a.inv_freq[j];
    const f32x2 turn = turn_of(kAxes ? (double)place : (double)pos_of[k], per_pos, a.rot_scale);
    cs[k][j] = turn[0];
    sn[k][j] = turn[1];
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
    norm_rope_row<T, D, kPairs>(
        x, ch, norm, !is_v, in, a.eps, a.rot_dim,
        [&](int j) __attribute__((always_inline)) {
          return j < 4 ? (is_q ? wq0[j & 3] : wk0[j & 3]) : (is_q ? wq1[j & 3] : wk1[j & 3]);
        },
        [&](const float *&ct, const float *&st) __attribute__((always_inline)) {
          ct = cs[tk];
          st = sn[tk];
        },
        [&]() __attribute__((always_inline)) { return base + tk * a.qkv_row + hd * D; },
        [&]() __attribute__((always_inline)) { return is_q ? a.q_w : a.k_w; });
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

template <typename T, int D, bool kCache, bool kAxes>
void run(const FrontArgs &a, bool interleaved, dim3 grid, hipStream_t stream) {
  const dim3 block(kFrontThreads);
  if (interleaved)
    hipLaunchKernelGGL((attn_front_kernel<T, D, Pairs::kInterleaved, kCache, kAxes>), grid, block, 0,
                       stream, a);
  else if (a.rot_dim % 8 == 0)
    hipLaunchKernelGGL((attn_front_kernel<T, D, Pairs::kHalf, kCache, kAxes>), grid, block, 0, stream,
                       a);
  else
    hipLaunchKernelGGL((attn_front_kernel<T, D, Pairs::kHalfOdd, kCache, kAxes>), grid, block, 0,
                       stream, a);
}

template <typename T, int D>
void run_of(const FrontArgs &a, bool interleaved, dim3 grid, hipStream_t stream) {
  if (a.positions)
    a.k_pages ? run<T, D, true, true>(a, interleaved, grid, stream)
              : run<T, D, false, true>(a, interleaved, grid, stream);
  else
    a.k_pages ? run<T, D, true, false>(a, interleaved, grid, stream)
              : run<T, D, false, false>(a, interleaved, grid, stream);
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
