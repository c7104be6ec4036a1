// ssm_pieces.h -- pieces of a row: kN neighbouring elements that are moved
// with 16-byte loads and stores wherever they start (gfx950 takes global
// accesses at any element's address), the row's last piece element by element
// where it is not whole, and sums over lanes.  Included by .hip sources only.
#pragma once

#include "ssm_device.h"

namespace ssm {
namespace dev {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

// kN (a multiple of 8 for bf16, of 4 for fp32) elements as they are in memory.
template <typename T, int kN>
struct Piece {
  static constexpr int kWords = kN * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      u32x4_t x;
      if constexpr (sizeof(T) == 2)
        x = *reinterpret_cast<const u32x4_a2 *>(p + 8 * i);
      else
        x = *reinterpret_cast<const u32x4_a4 *>(p + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * i + e] = x[e];
    }
  }
  // the first n of kN elements, 0 behind them
  __device__ __forceinline__ void load_some(const T *p, int n) {
    zero();
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (e < n) {
        if constexpr (sizeof(T) == 2)
          w[e / 2] |= static_cast<uint32_t>(p[e]) << (16 * (e % 2));
        else
          w[e] = __float_as_uint(p[e]);
      }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 2)
      return e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    else
      return __uint_as_float(w[e]);
  }
  __device__ __forceinline__ void set(const float (&v)[kN]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 2)
        w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      else
        w[i] = __float_as_uint(v[i]);
    }
  }
  __device__ __forceinline__ void store(T *p) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const u32x4_t x{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<u32x4_a2 *>(p + 8 * i) = x;
      else
        *reinterpret_cast<u32x4_a4 *>(p + 4 * i) = x;
    }
  }
  __device__ __forceinline__ void store_some(T *p, int n) const {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (e < n) {
        if constexpr (sizeof(T) == 2)
          p[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e % 2)));
        else
          p[e] = __uint_as_float(w[e]);
      }
  }
};

// Piece at element q * kN of a row of dim elements (q * kN < dim).
template <typename T, int kN>
__device__ __forceinline__ void load_piece(Piece<T, kN> &x, const T *row, int q, int dim) {
  const int left = dim - q * kN;
  if (left >= kN)
    x.load(row + q * kN);
  else
    x.load_some(row + q * kN, left);
}
template <typename T, int kN>
__device__ __forceinline__ void store_piece(T *row, int q, int dim, const float (&v)[kN]) {
  Piece<T, kN> x;
  x.set(v);
  const int left = dim - q * kN;
  if (left >= kN)
    x.store(row + q * kN);
  else
    x.store_some(row + q * kN, left);
}
template <typename T, int kN>
__device__ __forceinline__ void get_piece(const T *row, int q, int dim, float (&v)[kN]) {
  Piece<T, kN> x;
  load_piece(x, row, q, dim);
#pragma unroll
  for (int e = 0; e < kN; ++e) v[e] = x[e];
}

constexpr int kRowHalfMirror = 0x141;
constexpr int kRowMirror = 0x140;

// Sum over each group of `lanes` (8, 16, 32 or 64) neighbouring lanes, the
// same in every lane of the group: quads, halves and rows of 16 by DPP, rows
// by the lane-swap instructions.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  v += dpp<kQuadXor1>(0.0f, v);
  v += dpp<kQuadXor2>(0.0f, v);
  v += dpp<kRowHalfMirror>(0.0f, v);
  if (lanes >= 16) v += dpp<kRowMirror>(0.0f, v);
  if (lanes >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if (lanes >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

}  // namespace dev
}  // namespace ssm
