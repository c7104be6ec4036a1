// ssm_pieces.h -- pieces of a row: kN neighbouring elements that are moved
// with 16-byte loads and stores wherever they start (gfx950 takes global
// accesses at any element's address; 200 million elements copied from and to
// addresses that are no multiple of 4 took 3 % longer), and sums over lanes.
// Included by .hip sources only.
//
// A row's last piece, where the row does not fill it, ends with the row: its
// first elements belong to the piece before.  It is read whole, those elements
// are left out of sums, and only the others are written.  (Reading it element
// by element, one wait after another, cost rows of 8191 half of their time.)
#pragma once

#include "ssm_device.h"

namespace ssm {
namespace dev {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

// kN (a multiple of 4) elements as they are in memory.
template <typename T, int kN>
struct Piece {
  static constexpr int kWords = kN * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kWords == 2) {
      const u32x2_t x = *reinterpret_cast<const u32x2_a2 *>(p);
      w[0] = x[0];
      w[1] = x[1];
    }
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
  // a row of n < kN elements, in the last n places; the others repeat its first
  __device__ __forceinline__ void load_some(const T *p, int n) {
    T x[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int at = e - (kN - n);
      x[e] = p[at < 0 ? 0 : at];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 2)
        w[i] = x[2 * i] | static_cast<uint32_t>(x[2 * i + 1]) << 16;
      else
        w[i] = __float_as_uint(x[i]);
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
    if constexpr (kWords == 2) *reinterpret_cast<u32x2_a2 *>(p) = u32x2_t{w[0], w[1]};
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const u32x4_t x{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<u32x4_a2 *>(p + 8 * i) = x;
      else
        *reinterpret_cast<u32x4_a4 *>(p + 4 * i) = x;
    }
  }
  // the last n places, to p[0] and on
  __device__ __forceinline__ void store_some(T *p, int n) const {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (e >= kN - n) {
        if constexpr (sizeof(T) == 2)
          p[e - (kN - n)] = static_cast<uint16_t>(w[e / 2] >> (16 * (e % 2)));
        else
          p[e - (kN - n)] = __uint_as_float(w[e]);
      }
  }
};

// Whether place e of piece q belongs to it (and not to the one before, or to
// none): of a row of dim elements.
template <int kN>
__device__ __forceinline__ bool in_piece(int q, int e, int dim) {
  return e >= kN - (dim - q * kN);
}

// Piece q of a row of dim elements (q * kN < dim).
template <typename T, int kN>
__device__ __forceinline__ void load_piece(Piece<T, kN> &x, const T *row, int q, int dim) {
  if (dim >= kN) {
    const int at = q * kN;
    x.load(row + (at + kN <= dim ? at : dim - kN));
  } else {
    x.load_some(row, dim);
  }
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
