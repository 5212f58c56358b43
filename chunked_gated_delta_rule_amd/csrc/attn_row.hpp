// One head's row of q or k: RMS norm, weight, and the rotation of its first rot_dim
// channels, by the D / 8 lanes that own it, eight channels each. Shared by the kernels that
// write 16-bit rows (attn_front.hip) and 8-bit pages (attn_append8.hip).
#pragma once

#include <cfloat>
#include <type_traits>

#include "attn_common.hpp"

namespace gdn {

// How a lane's eight channels are placed: pairs inside the lane (half layout
// with rot_dim a multiple of 8, or interleaved), or (half layout with any other
// rot_dim) eight channels in a row whose partners are read one by one.
enum class Pairs { kHalf = 0, kInterleaved = 1, kHalfOdd = 2 };

// The least sum of squares that is taken as it is, and the factors for values whose sum is
// not fp32's (bf16 only): 2^128 2^-96 and 2^-126 2^96 have squares that are.
constexpr float kSmall = 0x1p-100f, kDown = 0x1p-96f, kUp = 0x1p96f;

// 1 / (2 pi), for angles counted in turns.
constexpr double kInvTwoPi = 0.15915494309189533577;

// cos and sin of position * per_pos radians, times `scale`. The angle is formed and reduced
// in 64 bits.
__device__ __forceinline__ f32x2 turn_of(double pos, float per_pos, float scale) {
  const double turns = pos * (double)per_pos * kInvTwoPi;
  const float f = (float)(turns - __builtin_rint(turns));  // -1/2 .. 1/2
  // cos(2 pi f), sin(2 pi f)
  return f32x2{scale * __builtin_amdgcn_cosf(f), scale * __builtin_amdgcn_sinf(f)};
}

template <typename T>
__device__ __forceinline__ void unpack4(const u32x2 &w, float *f) {
  f[0] = Elem<T>::lo(w[0]);
  f[1] = Elem<T>::hi(w[0]);
  f[2] = Elem<T>::lo(w[1]);
  f[3] = Elem<T>::hi(w[1]);
}

// A lane's channels: c0 .. c0 + 3 and c1 .. c1 + 3; whether they are turned (of the
// interleaved and odd layouts: some of them).
template <Pairs kPairs>
struct Channels {
  int c0, c1;
  bool turned;
  __device__ __forceinline__ Channels(int li, int rot_dim) {
    c0 = 8 * li;
    c1 = c0 + 4;
    turned = c0 < rot_dim;
    if constexpr (kPairs == Pairs::kHalf) {
      const int half = rot_dim >> 1;
      turned = li < half / 4;
      c0 = turned ? 4 * li : rot_dim + 8 * (li - half / 4);
      c1 = turned ? half + 4 * li : c0 + 4;
    }
  }
};

// x: a lane's channels of a row. norm: whether the row is normed; rot: whether it is
// turned. The rest is asked for where it is used, which keeps its addresses out of the
// registers: weight(j), of the lane's channel j; turns(ct, st), the cosines and sines of the
// row's pairs; and, where a pair's members lie in different lanes (and only with `in`),
// row(), the row in memory, and weights(), the head's (may be null). Every lane of the row
// takes part.
template <typename T, int D, Pairs kPairs, typename F, typename C, typename R, typename W>
__device__ __forceinline__ void norm_rope_row(float (&x)[8], const Channels<kPairs> &ch, bool norm,
                                              bool rot, bool in, float eps, int rot_dim,
                                              F weight, C turns, R row, W weights) {
  constexpr int kLanes = D / 8;  // lanes per head
  const int half = rot_dim >> 1;
  const int c0 = ch.c0;
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
  ss = sum16(ss);
  if constexpr (kLanes == 32) ss = sum16x(ss);
  float rn = norm ? 1.f / sqrtf(ss * (1.f / D) + eps) : 1.f;
  float by = 1.f;
  if constexpr (std::is_same_v<T, __bf16>) {
    // values whose squares leave fp32 (past about 2^60), or vanish in it with nothing
    // added to them, are brought to the middle of its range first
    const bool large = ss > FLT_MAX, small = ss < kSmall && eps < kSmall;
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
      if (norm) rn = 1.f / sqrtf(ss * (1.f / D) + eps * by * by);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] *= rn * weight(j);
    x[j + 4] *= rn * weight(j + 4);
  }
  if (rot) {
    const float *ct, *st;
    turns(ct, st);
    if constexpr (kPairs == Pairs::kHalf) {
      if (ch.turned) {
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
        if (c0 + 2 * j < rot_dim) {
          const float c = ct[(c0 >> 1) + j], d = st[(c0 >> 1) + j];
          const float u = x[2 * j], v = x[2 * j + 1];
          x[2 * j] = u * c - v * d;
          x[2 * j + 1] = v * c + u * d;
        }
      }
    } else {
      if (in) {
        // (formed ahead of the branch, the partners' addresses would take registers that six
        // waves per SIMD do not have: 8192 tokens of 40 heads of 128, rot_dim 34, from HBM 98 us
        // instead of 79)
        asm volatile("");
        const float *wp = weights();
        const T *values = row();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = c0 + j;
          if (c < rot_dim) {
            const bool low = c < half;
            const int p = low ? c + half : c - half, i = low ? c : p;
            const float y = static_cast<float>(values[p]) * by * rn * (wp ? wp[p] : 1.f);
            x[j] = x[j] * ct[i] + (low ? -y : y) * st[i];
          }
        }
      }
    }
  }
}

}  // namespace gdn
