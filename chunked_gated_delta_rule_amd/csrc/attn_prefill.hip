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

// Slots of the query tiles: sequence s starts at slot floor(cu[s] / kBM) + s,
// which is distinct for every tile of the batch and grows with s, so a slot's
// sequence is found by a search and no table is needed.
__host__ __device__ inline int64_t tile_slots(int64_t t_max, int64_t n_max) {
  return t_max / kBM + n_max;
}

// Head and tile slot of a work-group. The last (longest) tiles come first. With
// a multiple of 8 heads, neighbouring heads (which read the same keys) go to one
// XCD, whose L2 then holds their keys and values.
__device__ __forceinline__ void place(int wg, int h, int slots, int &head, int &slot) {
  if (h % 8 == 0) {
    const int per = h / 8, i = wg >> 3;
    head = (wg & 7) * per + i % per;
    slot = slots - 1 - i / per;
  } else {
    head = wg % h;
    slot = slots - 1 - wg / h;
  }
}

template <typename T, int D>
struct Tile {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kLoads = kBN * kRowBytes / 4096;  // per wave: 1 KB each
  static constexpr int kRowsPerLoad = 4096 / kRowBytes;  // of the work-group's four waves
  // Chunk (16 bytes) in which row r keeps its chunk c. For K, whose fragments
  // take one chunk of 32 rows, the rows differ in the low bits; for V, whose
  // transposing reads take four neighbouring chunks of four rows, in bits 2, 3.
  static __device__ __forceinline__ int k_swz(int r) { return r & 15; }
  static __device__ __forceinline__ int v_swz(int r) { return (r & 3) << 2; }
};

// Waits for this wave's copies into LDS. A barrier alone does not: its ordering
// covers the wave's own LDS accesses, not copies still in flight.
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Copies 64 rows (those of them that the descriptor's range holds, zeros for the
// others) straight to LDS: lane l of wave w fills the 16 bytes at 4096 i + 1024 w +
// 16 l with the chunk that belongs there.
template <typename T, int D, bool kV>
__device__ __forceinline__ void fetch(Lds<T> dst, rsrc_t src, int row_bytes, int lane, int w) {
  typedef Tile<T, D> L;
#pragma unroll
  for (int i = 0; i < L::kLoads; ++i) {
    const int in = 1024 * w + 16 * lane;
    const int row = i * L::kRowsPerLoad + in / L::kRowBytes, at = in % L::kRowBytes / 16;
    const int ch = at ^ (kV ? L::v_swz(row) : L::k_swz(row));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        src, (Lds<void>)(dst + 2048 * i + 512 * w), 16,
        row * row_bytes + 16 * ch, 0, 0, 0);
  }
}

// One query tile's running state, and its step over one tile of keys.
template <typename T, int D>
struct Rows {
  typedef typename Elem<T>::vec8 vec8;
  vec8 q[D / 16];
  f32x16 o[D / 32];
  float m, l;  // maximum (log2 scale) and this lane's part of the sum

  __device__ __forceinline__ void step(Lds<T> kt, Lds<T> vt, int k0, int lim, bool masked,
                                       float scale_log2, int lane) {
    typedef Tile<T, D> L;
    const int col = lane & 31, hh = lane >> 5;
    f32x16 sc[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
    const int kx = L::k_swz(col) ^ hh;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int at = col * D + 8 * ((2 * i) ^ kx);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        sc[t] = mfma32(*(Lds<const vec8>)(kt + at + 32 * t * D), q[i], sc[t]);
    }
    // order: eight fragments ahead, then products and reads in turn
    __builtin_amdgcn_sched_group_barrier(kSchedLds, D / 16, 0);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedLds, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, D / 16, 0);
    if (masked) {
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
    }
    const float ms = m == kNegInf ? 0.f : m;
    // lane's part of a transposing read: row 4 hh + (s16 >> 2) (+ 8), columns 32 i +
    // 16 gb + 4 (s16 & 3)
    const int s16 = lane & 15, gb = (lane >> 4) & 1, r0 = 4 * hh + (s16 >> 2);
    const int vx = L::v_swz(r0) ^ (2 * gb + ((s16 & 3) >> 1));
    // 16 keys at a time: the weights of the next are formed while the products
    // of these run
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t wd[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e0 = fast_exp2(fmaf(sc[b >> 1][8 * (b & 1) + 2 * i], scale_log2, -ms));
        const float e1 = fast_exp2(fmaf(sc[b >> 1][8 * (b & 1) + 2 * i + 1], scale_log2, -ms));
        l += e0 + e1;
        wd[i] = Elem<T>::pack(e0, e1);
      }
      const vec8 p = __builtin_bit_cast(vec8, u32x4{wd[0], wd[1], wd[2], wd[3]});
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int at = r0 * D + 4 * (s16 & 1) + 8 * ((4 * i) ^ vx);
        const u32x2 x = tr_read<T>(vt, at + 16 * b * D), y = tr_read<T>(vt, at + (16 * b + 8) * D);
        o[i] = mfma32(__builtin_bit_cast(vec8, u32x4{x[0], x[1], y[0], y[1]}), p, o[i]);
      }
    }
    // order: the first keys' fragments and weights, then under each product the
    // reads of a later one and a part of the next weights
    __builtin_amdgcn_sched_group_barrier(kSchedLds, D / 16, 1);
    __builtin_amdgcn_sched_group_barrier(kSchedValu, 28, 1);
#pragma unroll
    for (int i = 0; i < D / 8 - D / 32; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedLds, 2, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 7, 1);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, D / 32, 1);
  }
};

template <typename T, int D>
__global__ __launch_bounds__(256, D == 128 ? 2 : 1) void attn_prefill_kernel(PrefillArgs a,
                                                                            int slots) {
  // four arrays of their own, so that a tile in flight is known to be another
  // than the ones being read
  __shared__ __attribute__((aligned(16))) T k_a[kBN * D], v_a[kBN * D], k_b[kBN * D], v_b[kBN * D];

  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  const int wg = flat_block();
  int head, slot;
  place(wg, a.h, slots, head, slot);
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

  Rows<T, D> x;
  {
    const T *qp = static_cast<const T *>(a.q) + (int64_t)(qb + r) * a.q_row + head * D + 8 * hh;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      x.q[i] = *reinterpret_cast<const typename Rows<T, D>::vec8 *>(qp + 16 * i);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) x.o[i][j] = 0.f;
  x.m = kNegInf;
  x.l = 0.f;

  const T *kp = static_cast<const T *>(a.k) + (int64_t)kb * a.k_row + kvh * D;
  const T *vp = static_cast<const T *>(a.v) + (int64_t)kb * a.v_row + kvh * D;
  const int k_bytes = (int)a.k_row * 2, v_bytes = (int)a.v_row * 2;
  // a tile's rows as a range that ends with the sequence's last key
  auto get = [&](int j, Lds<T> kt, Lds<T> vt) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)j * kBN;
    const int rows = min(kBN, lk - (int)k0);
    fetch<T, D, false>(kt, make_rsrc(kp + k0 * a.k_row, (rows - 1) * k_bytes + D * 2), k_bytes, lane, w);
    fetch<T, D, true>(vt, make_rsrc(vp + k0 * a.v_row, (rows - 1) * v_bytes + D * 2), v_bytes, lane, w);
  };
  auto step = [&](int j, Lds<T> kt, Lds<T> vt) __attribute__((always_inline)) {
    const int k0 = j * kBN;
    if (k0 <= wave_hi) x.step(kt, vt, k0, lim, k0 + kBN - 1 > wave_lo, a.scale_log2, lane);
  };
  auto L = [](T *p) { return (Lds<T>)p; };
  if (tiles > 0) get(0, L(k_a), L(v_a));
  for (int j = 0; j < tiles; j += 2) {
    wait_copies();
    __syncthreads();  // tile j is there, and the other pair is no longer read
    if (j + 1 < tiles) get(j + 1, L(k_b), L(v_b));
    step(j, L(k_a), L(v_a));
    if (j + 1 >= tiles) break;
    wait_copies();
    __syncthreads();
    if (j + 2 < tiles) get(j + 2, L(k_a), L(v_a));
    step(j + 1, L(k_b), L(v_b));
  }

  const float l = sum32(x.l);
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees no key gives zeros
  if (r0 + col >= lq) return;
  T *op = static_cast<T *>(a.o) + ((int64_t)(qb + r0 + col) * a.h + head) * D + 4 * hh;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<u32x2 *>(op + 32 * i + 8 * b) =
          u32x2{Elem<T>::pack(x.o[i][4 * b] * inv, x.o[i][4 * b + 1] * inv),
                Elem<T>::pack(x.o[i][4 * b + 2] * inv, x.o[i][4 * b + 3] * inv)};
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
