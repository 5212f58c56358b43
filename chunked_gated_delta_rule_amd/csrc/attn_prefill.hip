// Causal attention over packed prompts (grouped heads, queries the last tokens
// of their keys), forward:  o_r = sum_{c <= lim(r)} softmax_c(scale q_r . k_c) v_c.
//
// One pass over the keys per query tile with a running maximum and sum per row.
// A 256-thread work-group (four waves) owns 128 query rows of one head, 32 per
// wave, and walks the keys 64 at a time; K and V tiles go through LDS, double
// buffered, and are shared by the four waves. Everything else stays in the
// wave's registers: scores are formed transposed, S^T = K Q^T, so a lane's
// column is one query row and the softmax statistics are per lane (one
// exchange between the two half-waves per tile), and the C layout of S^T is,
// with the keys taken in the order the accumulator holds them, the B operand
// of O^T += V^T P^T. V^T comes from the row-major tile with transposing LDS
// reads. So the scores and weights never touch LDS.
//
// LDS rows are swizzled by 16-byte chunk (chunk ^ (row & 15)): the 32 rows a
// K fragment reads at one chunk, and the rows a transposing read spans, fall
// into different banks.
#include "attn_common.hpp"
#include "attn_launch.hpp"

namespace gdn {

namespace {

constexpr int kBM = 128;  // query rows per work-group
constexpr int kBN = 64;   // keys per tile

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Transposing read: within each 16-lane group, lane s supplies four elements
// of row (s >> 2), columns 4 (s & 3) .., and lane j receives column j of the
// four rows.
__device__ __forceinline__ u32x2 tr_read(const void *p) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(const_cast<void *>(p))));
}

// Slots of the query tiles: sequence s starts at slot floor(cu[s] / kBM) + s,
// which is distinct for every tile of the batch and grows with s, so a slot's
// sequence is found by a search and no table is needed.
__host__ __device__ inline int64_t tile_slots(int64_t t_max, int64_t n_max) {
  return t_max / kBM + n_max;
}

template <typename T, int D>
__global__ __launch_bounds__(256, D == 128 ? 2 : 1) void attn_prefill_kernel(PrefillArgs a,
                                                                            int slots) {
  typedef typename Elem<T>::vec8 vec8;
  constexpr int kCh = D / 8;                  // 16-byte chunks per row
  constexpr int kStage = kBN * kCh / 256;     // chunks per thread and tile
  __shared__ __attribute__((aligned(16))) T lds[2][2][kBN * D];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int col = lane & 31, hh = lane >> 5;
  // heads fastest, the last (longest) tiles first
  const int wg = flat_block();
  const int head = wg % a.h, slot = slots - 1 - wg / a.h;
  if (slot < 0) return;  // past the grid's count (last row)
  const int s = wave_search(a.n_max, slot, lane,
                            [&](int i) { return cu_at(a.cu_q, i, a.t_max) / kBM + i; });
  const int qb = cu_at(a.cu_q, s, a.t_max), lq = cu_end(a.cu_q, s, qb, a.t_max) - qb;
  const int q0 = (slot - (qb / kBM + s)) * kBM;
  if (q0 < 0 || q0 >= lq) return;  // no tile of the sequence has this slot
  const int kb = cu_at(a.cu_k, s, a.tk_max), lk = cu_end(a.cu_k, s, kb, a.tk_max) - kb;
  const int kvh = head / (a.h / a.hkv);
  const int past = lk - lq;  // row r sees keys 0 .. past + r

  const int r0 = q0 + 32 * w;                  // the wave's first row
  const int r = min(r0 + col, lq - 1);         // this lane's row (the last one again past the end)
  const int lim = past + r;
  const int wave_lo = past + min(r0, lq - 1), wave_hi = past + min(r0 + 31, lq - 1);
  const int keys = min(past + min(q0 + kBM, lq), lk);  // keys any row of the tile sees
  const int tiles = keys > 0 ? (keys + kBN - 1) / kBN : 0;

  vec8 qf[D / 16];
  {
    const T *qp = static_cast<const T *>(a.q) + (int64_t)(qb + r) * a.q_row + head * D + 8 * hh;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) qf[i] = *reinterpret_cast<const vec8 *>(qp + 16 * i);
  }
  const T *kp = static_cast<const T *>(a.k) + (int64_t)kb * a.k_row + kvh * D;
  const T *vp = static_cast<const T *>(a.v) + (int64_t)kb * a.v_row + kvh * D;

  u32x4 ks[kStage], vs[kStage];
  auto load = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int idx = i * 256 + tid, row = min(k0 + idx / kCh, lk - 1), ch = idx % kCh;
      ks[i] = *reinterpret_cast<const u32x4 *>(kp + (int64_t)row * a.k_row + 8 * ch);
      vs[i] = *reinterpret_cast<const u32x4 *>(vp + (int64_t)row * a.v_row + 8 * ch);
    }
  };
  auto stage = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int idx = i * 256 + tid, row = idx / kCh, ch = idx % kCh;
      const int at = row * D + 8 * (ch ^ (row & 15));
      *reinterpret_cast<u32x4 *>(&lds[buf][0][at]) = ks[i];
      *reinterpret_cast<u32x4 *>(&lds[buf][1][at]) = vs[i];
    }
  };

  f32x16 o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  float m = kNegInf, l = 0.f;  // maximum (log2 scale) and this lane's part of the sum

  if (tiles > 0) {
    load(0);
    stage(0);
  }
  __syncthreads();
  for (int j = 0; j < tiles; ++j) {
    const int k0 = j * kBN, buf = j & 1;
    if (j + 1 < tiles) load(k0 + kBN);
    if (k0 <= wave_hi) {
      f32x16 sc[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
        const int row = 32 * t + col;
        const T *base = &lds[buf][0][row * D];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const vec8 kf = *reinterpret_cast<const vec8 *>(base + 8 * ((2 * i + hh) ^ (row & 15)));
          sc[t] = mfma32(kf, qf[i], sc[t]);
        }
      }
      if (k0 + kBN - 1 > wave_lo) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sc[t][i] = k0 + 32 * t + 8 * (i >> 2) + 4 * hh + (i & 3) <= lim ? sc[t][i] : kNegInf;
      }
      float mx = kNegInf;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[t][i]);
      mx = fmaxf(mx, swap32(mx)) * a.scale_log2;
      if (__any(mx > m + kRescaleLog2)) {
        const float mn = fmaxf(m, mx);
        const float al = mn == kNegInf ? 1.f : fast_exp2(m - mn);
        m = mn;
        l *= al;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k) o[i][k] *= al;
      }
      const float ms = m == kNegInf ? 0.f : m;
      vec8 p[4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t wd[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e0 = fast_exp2(fmaf(sc[t][8 * b + 2 * i], a.scale_log2, -ms));
            const float e1 = fast_exp2(fmaf(sc[t][8 * b + 2 * i + 1], a.scale_log2, -ms));
            l += e0 + e1;
            wd[i] = Elem<T>::pack(e0, e1);
          }
          p[2 * t + b] = __builtin_bit_cast(vec8, u32x4{wd[0], wd[1], wd[2], wd[3]});
        }
      const T *vt = lds[buf][1];
      const int s16 = lane & 15, gb = (lane >> 4) & 1;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int ch = 4 * i + 2 * gb + ((s16 & 3) >> 1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int ra = 16 * b + 4 * hh + (s16 >> 2), rb = ra + 8;
          const u32x2 x = tr_read(vt + ra * D + 8 * (ch ^ (ra & 15)) + 4 * (s16 & 1));
          const u32x2 y = tr_read(vt + rb * D + 8 * (ch ^ (rb & 15)) + 4 * (s16 & 1));
          o[i] = mfma32(__builtin_bit_cast(vec8, u32x4{x[0], x[1], y[0], y[1]}), p[b], o[i]);
        }
      }
    }
    if (j + 1 < tiles) stage(buf ^ 1);
    __syncthreads();
  }

  l += swap32(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees no key gives zeros
  if (r0 + col >= lq) return;
  T *op = static_cast<T *>(a.o) + ((int64_t)(qb + r0 + col) * a.h + head) * D + 4 * hh;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<u32x2 *>(op + 32 * i + 8 * b) =
          u32x2{Elem<T>::pack(o[i][4 * b] * inv, o[i][4 * b + 1] * inv),
                Elem<T>::pack(o[i][4 * b + 2] * inv, o[i][4 * b + 3] * inv)};
}

}  // namespace

hipError_t launch_attn_prefill(const gdn_attn_config *cfg, PrefillArgs a, hipStream_t stream) {
  if (cfg->t_max == 0) return hipSuccess;
  const int64_t slots = tile_slots(cfg->t_max, cfg->n_max);
  dim3 grid;
  if (!flat_grid(slots * cfg->h, 256, grid)) return hipErrorInvalidValue;
  const dim3 block(256);
  const int n = static_cast<int>(slots);
  if (cfg->dtype == GDN_BF16) {
    if (cfg->d == 128)
      hipLaunchKernelGGL((attn_prefill_kernel<__bf16, 128>), grid, block, 0, stream, a, n);
    else
      hipLaunchKernelGGL((attn_prefill_kernel<__bf16, 256>), grid, block, 0, stream, a, n);
  } else {
    if (cfg->d == 128)
      hipLaunchKernelGGL((attn_prefill_kernel<_Float16, 128>), grid, block, 0, stream, a, n);
    else
      hipLaunchKernelGGL((attn_prefill_kernel<_Float16, 256>), grid, block, 0, stream, a, n);
  }
  return hipGetLastError();
}

}  // namespace gdn
