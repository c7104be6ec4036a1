// ssm_linattn_core.h -- the chunk kernel of linear attention with a decay for
// each head on gfx950's matrix cores.  Included by the .hip files that
// instantiate it.
//
// With the recurrence S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = S_t^T q_t and
// a_t the sum of g from the chunk's start to t, a chunk of T tokens is
//   o_t = e^{a_t} S_in^T q_t + sum_{s<=t} e^{a_t - a_s} (q_t . k_s) v_s
//   S_out = e^{a_T} S_in + sum_s e^{a_T - a_s} k_s v_s^T.
// Its gradients are the same products with other operands.  With M the
// adjoint of the state that leaves the chunk:
//   dq: in token order, (q, k, v) := (do, v, k), state S^T
//   dv: against it,     (q, k, v) := (k, q, do), state M
//   dk: against it,     (q, k, v) := (v, do, q), state M^T
// where against token order s runs over s >= t, the weights are e^{a_s - a_t}
// inside the chunk, e^{a_T - a_t} on the state and e^{a_s} into it.  So one
// kernel serves the forward pass, the three gradients and the pass that
// forms only the states of the segments.
//
// The decay sums run in 64 bits and every weight is the exponential of a
// difference, so that a strong decay (even -inf, a reset) neither
// overflows nor cancels.
#pragma once

#include <type_traits>

#include "ssm_device.h"
#include "ssm_linattn_internal.h"

namespace ssm {
namespace lin {

using namespace dev;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A fragment: 8 elements of the contracted index a lane holds for one row
// (or column) of a 16 x 16 product over 32: lane l, element e belong to
// row l % 16 and contracted position 8 * (l / 16) + e.  In 32 bits the
// product is 8 steps of 4, step e taking element e of every lane.
template <typename T> struct Traits;
template <> struct Traits<uint16_t> {
  typedef bf16x8 Frag;
  typedef bf16x4 Half;
  typedef __bf16 Elem;
  static constexpr int kChunk = kLinChunkBf16;
  typedef float Sum;  // of decays, where two are subtracted for a pair's weight
  static constexpr bool kBf16 = true;
};
template <> struct Traits<float> {
  typedef f32x8 Frag;
  typedef f32x4 Half;
  typedef float Elem;
  static constexpr int kChunk = kLinChunkF32;
  typedef double Sum;
  static constexpr bool kBf16 = false;
};

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

// Elements p[0..3] and p[16..19]: the fragment whose contracted positions
// are the rows a lane holds of two stacked 16-row accumulator tiles.
__device__ __forceinline__ bf16x8 two_halves(const __bf16 *p) {
  const bf16x4 a = *reinterpret_cast<const bf16x4 *>(p);
  const bf16x4 b = *reinterpret_cast<const bf16x4 *>(p + 16);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x8 two_halves(const float *p) {
  const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
  const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 16);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Fragment of a row-major [position][column] LDS tile contracted over its
// rows, `row` to `row` + 31: lane l gets column col + l % 16, and in elements
// 0..3 the positions row + 4 * (l / 16) + e, in 4..7 those 16 further on (the
// order of two_halves).  In bf16 the transposing LDS read hands every lane of
// 16 one column of the 4 x 16 block that the 16 lanes address; 32 lanes read
// 8 neighbouring rows at once, which lie 8 banks apart (measured: 2 cycles, as
// without conflicts).
template <int kStride>
__device__ __forceinline__ bf16x8 frag_by_column(const __bf16 *tile, int row, int col, int lane) {
  const int li = lane & 15, lq = lane >> 4;
  const __bf16 *p = tile + (row + 4 * lq + (li >> 2)) * kStride + col + 4 * (li & 3);
  typedef __attribute__((address_space(3))) s16x4 *Lds;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 16 * kStride));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int kStride>
__device__ __forceinline__ f32x8 frag_by_column(const float *tile, int row, int col, int lane) {
  const float *p = tile + (row + 4 * (lane >> 4)) * kStride + col + (lane & 15);
  f32x8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = p[(e % 4 + e / 4 * 16) * kStride];
  return r;
}

__device__ __forceinline__ bf16x8 to_frag(f32x8 v, bf16x8) {
  return __builtin_convertvector(v, bf16x8);
}
__device__ __forceinline__ f32x8 to_frag(f32x8 v, f32x8) { return v; }

// What is left of v behind hi, as two more bf16 values: with hi 24 bits, those
// of fp32.
__device__ __forceinline__ void split(f32x8 v, bf16x8 hi, bf16x8 *mid, bf16x8 *lo) {
  const f32x8 rest = v - __builtin_convertvector(hi, f32x8);
  *mid = to_frag(rest, bf16x8{});
  *lo = to_frag(rest - __builtin_convertvector(*mid, f32x8), bf16x8{});
}
__device__ __forceinline__ void split(f32x8, f32x8, f32x8 *, f32x8 *) {}

// The same value, unknown to the compiler: what is computed from it is made
// anew where it is used, not kept in registers from chunk to chunk.
__device__ __forceinline__ int anew(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The value, known to be the same in every lane, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Where a segment lies.
struct Segment {
  int64_t begin, end;  // token rows
  int seq;
  int seg;             // its number in the sequence
  bool last;           // of its sequence
  bool real;           // the slot is in use
};

__device__ __forceinline__ int64_t cu_at(const LinPlan &p, int i) {
  const int64_t c = p.cu[i];
  return c < 0 ? 0 : c > p.tokens ? p.tokens : c;
}

// Rows of a sequence; offsets outside [0, tokens], or that fall, are brought
// into range, so that no offset reaches memory outside the arrays.
__device__ __forceinline__ void sequence_rows(const LinPlan &p, int seq, int64_t *begin,
                                              int64_t *end) {
  if (!p.cu) {
    *begin = seq * p.seqlen;
    *end = *begin + p.seqlen;
    return;
  }
  const int64_t b = cu_at(p, seq), e = cu_at(p, seq + 1);
  *begin = b;
  *end = e < b ? b : e;
}

__device__ __forceinline__ int64_t first_slot(const LinPlan &p, int seq) {
  return p.cu ? cu_at(p, seq) / p.seg_len + seq : seq * p.segs;
}

__device__ __forceinline__ Segment segment_of(const LinPlan &p, int64_t slot) {
  Segment s;
  if (!p.cu) {
    s.seq = static_cast<int>(slot / p.segs);
  } else {
    int lo = 0, hi = p.nseq - 1;  // the last sequence whose first slot is <= slot
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_slot(p, mid) <= slot) lo = mid;
      else hi = mid - 1;
    }
    s.seq = lo;
  }
  s.seq = __builtin_amdgcn_readfirstlane(s.seq);
  s.seg = __builtin_amdgcn_readfirstlane(static_cast<int>(slot - first_slot(p, s.seq)));
  int64_t b, e;
  sequence_rows(p, s.seq, &b, &e);
  b = uniform(b);
  e = uniform(e);
  s.begin = b + s.seg * p.seg_len;
  // an empty sequence has one (empty) segment, which hands its state on
  s.real = s.seg >= 0 && (s.begin < e || s.seg == 0);
  s.end = s.begin + p.seg_len < e ? s.begin + p.seg_len : e;
  s.last = s.end == e;
  return s;
}

// log2 of a token's decay factor: g / ln 2, no less than -256 (whose
// exponential is 0 in 32 bits: -inf must not meet itself in a difference).
__device__ __forceinline__ double log2_decay(float g) {
  const double x = static_cast<double>(g) * 1.4426950408889634;
  return x < -256.0 ? -256.0 : x;
}

__device__ __forceinline__ float decay_at(const float *g, int kind, int64_t t, int heads, int h) {
  return kind == kLinDecayNone ? 0.0f : kind == kLinDecayHead ? g[h] : g[t * heads + h];
}

// Inclusive sums over the first kWidth lanes of a wave.
template <int kWidth>
__device__ __forceinline__ double wave_sums(double v, int lane) {
#pragma unroll
  for (int d = 1; d < kWidth; d *= 2) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Byte view of `rows` token rows (wave-uniform) for buffer loads: what lies
// behind the last row's end reads as 0.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_view(const T *base, int64_t stride,
                                                            int rows, int d) {
  const int bytes = rows > 0 ? static_cast<int>(((rows - 1) * stride + d) * sizeof(T)) : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(base), 0, bytes, kBufferWord3);
}

constexpr float kLargest = 3.4028235e38f;  // finite

constexpr int kNowhere = 0x7ffffff0;  // behind the end of every view

// kRows token rows of one head, kCols elements wide in LDS (the head's d,
// zeros behind), from memory to registers in pieces of 16 bytes.  Byte
// offsets are the same for every chunk; rows behind the sequence's end lie
// behind the view.  Without kVec the pieces are put together from elements.
template <typename T, int kRows, int kCols, int kThreads, bool kVec>
struct Tile {
  static constexpr int kPer = 16 / sizeof(T);           // elements of a piece
  static constexpr int kRowPieces = kCols / kPer;
  static constexpr int kPieces = kRows * kRowPieces / kThreads;
  static_assert(kRows * kRowPieces % kThreads == 0, "whole pieces per thread");
  static_assert(kThreads % kRowPieces == 0, "a thread's pieces are in one column");
  u32x4 r[kPieces];

  __device__ __forceinline__ void load(const T *base, int64_t stride, int rows, int d, int tid) {
    const __amdgpu_buffer_rsrc_t v = rows_view(base, stride, rows, d);
    const int c = tid % kRowPieces * kPer;
    const int row_bytes = static_cast<int>(stride * sizeof(T));
    // (past kNowhere the offsets stay, unsigned, behind every view)
    const unsigned off0 = c < d ? tid / kRowPieces * row_bytes + c * sizeof(T) : kNowhere;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int off = static_cast<int>(off0 + static_cast<unsigned>(i * (kThreads / kRowPieces)) * row_bytes);
      if constexpr (kVec) {
        r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(v, off, 0, 0));
      } else {
        const int left = d - c;  // elements of the row from here
        if constexpr (sizeof(T) == 2) {
          uint32_t e[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            e[k] = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(
                v, k < left ? off + 2 * k : kNowhere, 0, 0));
#pragma unroll
          for (int k = 0; k < 4; ++k) r[i][k] = e[2 * k] | (e[2 * k + 1] << 16);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            r[i][k] = __builtin_amdgcn_raw_buffer_load_b32(
                v, k < left ? off + 4 * k : kNowhere, 0, 0);
        }
      }
    }
  }

  template <int kStride>
  __device__ __forceinline__ void store(typename Traits<T>::Elem *tile, int tid) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int q = tid + kThreads * i, row = q / kRowPieces, c = (q % kRowPieces) * kPer;
      *reinterpret_cast<u32x4 *>(tile + row * kStride + c) = r[i];
    }
  }
};

// 4 neighbouring elements at a byte offset of a view, n of them in the row,
// as they are in memory.
template <typename T, bool kVec>
struct Four {
  uint32_t w[sizeof(T)];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t v, int off, int n) {
    if constexpr (kVec && sizeof(T) == 2) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(v, n > 0 ? off : kNowhere, 0, 0);
      w[0] = x[0];
      w[1] = x[1];
    } else if constexpr (kVec) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b128(v, n > 0 ? off : kNowhere, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = x[e];
    } else if constexpr (sizeof(T) == 2) {
      uint32_t x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = static_cast<uint16_t>(
            __builtin_amdgcn_raw_buffer_load_b16(v, e < n ? off + 2 * e : kNowhere, 0, 0));
      w[0] = x[0] | (x[1] << 16);
      w[1] = x[2] | (x[3] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = __builtin_amdgcn_raw_buffer_load_b32(v, e < n ? off + 4 * e : kNowhere, 0, 0);
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 2)
      return e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    else
      return __builtin_bit_cast(float, w[e]);
  }
};

// A fragment straight from memory: 8 elements at a byte offset of a view,
// `left` of them in the row.
template <typename T, bool kVec>
__device__ __forceinline__ typename Traits<T>::Frag view_frag(__amdgpu_buffer_rsrc_t v, int off,
                                                              int left) {
  typedef typename Traits<T>::Frag Frag;
  if constexpr (sizeof(T) == 2) {
    if constexpr (kVec) {
      return __builtin_bit_cast(
          Frag, __builtin_amdgcn_raw_buffer_load_b128(v, left > 0 ? off : kNowhere, 0, 0));
    } else {
      typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
      u16x8 x;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = __builtin_amdgcn_raw_buffer_load_b16(v, e < left ? off + 2 * e : kNowhere, 0, 0);
      return __builtin_bit_cast(Frag, x);
    }
  } else {
    Frag f;
    if constexpr (kVec) {
      const f32x4 a = __builtin_bit_cast(
          f32x4, __builtin_amdgcn_raw_buffer_load_b128(v, left > 0 ? off : kNowhere, 0, 0));
      const f32x4 b = __builtin_bit_cast(
          f32x4, __builtin_amdgcn_raw_buffer_load_b128(v, left > 4 ? off + 16 : kNowhere, 0, 0));
      f = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            v, e < left ? off + 4 * e : kNowhere, 0, 0));
    }
    return f;
  }
}

// Stores 4 neighbouring elements at a byte offset of a view, n of them in
// the row.  (A store behind the view is dropped.)
template <bool kVec>
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t v, int off, f32x4 x, int n,
                                       uint16_t) {
  if constexpr (kVec) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(
        u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])}, v, n > 0 ? off : kNowhere, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __builtin_amdgcn_raw_buffer_store_b16(from_f32<uint16_t>(x[e]), v,
                                            e < n ? off + 2 * e : kNowhere, 0, 0);
  }
}
template <bool kVec>
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t v, int off, f32x4 x, int n, float) {
  if constexpr (kVec) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), v,
                                           n > 0 ? off : kNowhere, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[e]), v,
                                            e < n ? off + 4 * e : kNowhere, 0, 0);
  }
}

// One workgroup: kWaves waves, one segment of kHeads heads that share k (and
// q), kCols output columns of each.  A wave owns 16 columns of the output and
// of the state of one head, and that kDK x 16 part of the state stays in its
// accumulator registers from chunk to chunk (the state tiles are the second
// operand of the next product as they stand: the first operand is read with
// its columns in the order the accumulators hold the rows).  The products are
// set up so that a lane holds 4 neighbouring output columns of one token.
// Per chunk: the tiles go from registers (loaded during the chunk before) to
// LDS; the waves share out the token pairs' products, each then takes all of
// them for its columns.
//
// Why so: every operand is read from memory once (q and k once for two heads,
// or once for each 128 columns), and neither the states inside a segment nor
// the pairs ever leave the CU.  Two workgroups of 8 waves fill a CU's
// registers.  What bounds it: no unit alone.  In the output pass the vector
// units issue 36 % of the time (530 vector instructions -- weights, packing,
// splitting, addresses -- against 80 matrix ones a wave and chunk), LDS works
// 37 % (a third of it bank conflicts; the states' pass has none), the matrix
// cores 18 %, and the waves wait 56 % of their cycles: the phases of a chunk
// follow one another, with two barriers.  Measured, bf16 (kernel trace, median
// over inputs in turn):
//   2 x 4096 tokens, 80 heads of 64 on states of 128, one q and k: output
//   pass 117 us (180 MB, 1.5 TB/s; 32 GFLOP, 276 TFLOP/s), states 52 us;
//   65536 tokens, 8 heads of 128 on 128: 163 us (537 MB, 3.3 TB/s), states 80 us;
//   24 prompts of 16384 tokens together, 16 heads of 128 on 128: 118 and 45 us.
// Tiles of 4 waves, 2 columns of tiles a wave, or the next chunk's loads
// behind the products were all slower.
//
// bf16 roundings: the weighted pair products and the state where it is an
// operand, once each (2^-8 of each term, as the output's own rounding); what
// goes into the state enters as three bf16 values, 24 bits of it, since the
// state is returned in 32 bits and is carried over the sequence (with two,
// 16 bits, the final state and the decay's gradient were off by 2.6e-6 and
// 1e-5 in the norm); likewise the state itself where dot products in 32 bits
// are wanted (kLinOutDot).
// The sums of decays, at most 2^14 in size, are subtracted in 32 bits for
// the weights of the pairs in bf16 (2^-10 at the largest sizes, a quarter of
// the rounding the product then has), else in 64.
template <typename T, int kDK, int kWaves, int kHeads, int kMode>
struct CoreShared {
  typedef Traits<T> Tr;
  typedef typename Tr::Elem Elem;
  static constexpr int C = Tr::kChunk, kCols = 16 * kWaves / kHeads;
  static constexpr bool kOut = kMode != kLinState;
  // row strides: 8 banks apart for the transposing reads and those of 16
  // bytes, 4 for those of 8 bytes (cycles a read, measured: 2 and 4, with the
  // other stride 4 and 8); q is read both ways
  static constexpr int kRowQ = kDK + (Tr::kBf16 ? 8 : 4), kRowK = kDK + (Tr::kBf16 ? 16 : 4);
  static constexpr int kRowV = kCols + (Tr::kBf16 ? 16 : 4), kRowP = C + (Tr::kBf16 ? 8 : 4);
  alignas(16) Elem Qs[kOut ? C * kRowQ : 8];
  alignas(16) Elem Ks[C * kRowK];
  alignas(16) Elem Vs[kHeads][C * kRowV];
  alignas(16) Elem Ps[kHeads][kOut ? C * kRowP : 8];
  typename Tr::Sum As[kHeads][C];      // sums of decays (log2)
  alignas(16) float Wi[kHeads][C];     // weights into,
  float Wo[kHeads][C];                 // out of the state
  float Wd[kHeads];                    // the chunk's decay
  float Dots[kMode == kLinOutDot ? kWaves * C : 1];
};

template <typename T, int kDK, int kWaves, int kHeads, int kMode, bool kRev, bool kVec>
__device__ __forceinline__ void core(const LinCore &p, unsigned block,
                                     CoreShared<T, kDK, kWaves, kHeads, kMode> &sm) {
  typedef Traits<T> Tr;
  typedef typename Tr::Frag Frag;
  typedef typename Tr::Elem Elem;
  typedef typename Tr::Sum Sum;
  typedef CoreShared<T, kDK, kWaves, kHeads, kMode> Shared;
  constexpr int C = Tr::kChunk, kNT = C / 16, kTS = C / 32;
  constexpr int kKS = kDK / 32, kIT = kDK / 16;
  constexpr int kThreads = 64 * kWaves, kCols = Shared::kCols;
  constexpr bool kBf16 = Tr::kBf16;
  constexpr bool kOut = kMode != kLinState, kDot = kMode == kLinOutDot;
  constexpr int kRowQ = Shared::kRowQ, kRowK = Shared::kRowK;
  constexpr int kRowV = Shared::kRowV, kRowP = Shared::kRowP;
  auto &Qs = sm.Qs;
  auto &Ks = sm.Ks;
  auto &Vs = sm.Vs;
  auto &Ps = sm.Ps;
  auto &As = sm.As;
  auto &Wi = sm.Wi;
  auto &Wo = sm.Wo;
  auto &Wd = sm.Wd;
  auto &Dots = sm.Dots;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const unsigned slices = (p.v.d + kCols - 1) / kCols;
  const unsigned teams = static_cast<unsigned>(p.plan.heads) / kHeads;
  const int slice = block % slices;
  const int h0 = block / slices % teams * kHeads;
  const int64_t slot = block / (slices * teams);
  const Segment sg = segment_of(p.plan, slot);
  if (!sg.real) return;
  const bool ends = kRev ? sg.seg == 0 : sg.last;  // nothing comes after it
  if (kMode == kLinState && ends) return;

  const int mine = kHeads == 1 ? 0 : wave / (kWaves / kHeads);  // this wave's head
  const int h = h0 + mine;
  const int j0 = slice * kCols;
  const int dk = p.k.d, dv = p.v.d - j0;     // columns from this slice's first
  const int64_t n = sg.end - sg.begin;
  const int chunks = static_cast<int>((n + C - 1) / C);
  const T *qh = static_cast<const T *>(p.q.p) + (h0 / p.q.div) * p.q.d;
  const T *kh = static_cast<const T *>(p.k.p) + (h0 / p.k.div) * p.k.d;

  // the state: tile it, element e is S[16 it + 4 lq + e][jw + li]
  const int jw = 16 * (kHeads == 1 ? wave : wave % (kWaves / kHeads));
  f32x4 S[kIT];
  const int64_t size = static_cast<int64_t>(p.k.d) * p.v.d;
  const int64_t by_slot = (slot * p.plan.heads + h) * size;
  const int64_t by_seq = (static_cast<int64_t>(sg.seq) * p.plan.heads + h) * size;
  auto state_view = [&](const float *at) __attribute__((always_inline)) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(at), 0,
                                             static_cast<int>(size * sizeof(float)), kBufferWord3);
  };
  // byte offset of an element of this lane's, from that of its first one
  auto state_off = [&](int first_off, int it, int e) __attribute__((always_inline)) {
    const int off = first_off + 4 * (16 * it + e) * p.sa;
    const bool in = 16 * it + 4 * lq + e < dk && jw + li < dv;
    return in ? off : kNowhere;
  };
  const int state0 = 4 * (4 * lq * p.sa + (j0 + jw + li) * p.sb);
  {
    const float *in = nullptr;
    const bool begins = kRev ? sg.last : sg.seg == 0;  // nothing comes before it
    if (kMode != kLinState)
      in = !begins ? p.in_slots + by_slot : p.in_seqs ? p.in_seqs + by_seq : nullptr;
#pragma unroll
    for (int it = 0; it < kIT; ++it) S[it] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (in) {
      const __amdgpu_buffer_rsrc_t v = state_view(in);
#pragma unroll
      for (int it = 0; it < kIT; ++it)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[it][e] = __uint_as_float(
              __builtin_amdgcn_raw_buffer_load_b32(v, state_off(state0, it, e), 0, 0));
    }
  }
  auto save = [&](float *out) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t v = state_view(out);
    const int at = anew(state0);
#pragma unroll
    for (int it = 0; it < kIT; ++it)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[it][e]), v, state_off(at, it, e), 0, 0);
  };
  // the decay's gradient needs the state before a sequence's last chunk
  constexpr bool kBeforeLast = kDot && !kRev;
  // the first wave of each head forms its weights
  const bool weighs = kHeads == 1 ? wave == 0 : wave % (kWaves / kHeads) == 0;
  double total = 0.0;  // state pass: the segment's sum of decays (those waves)

  Tile<T, C, kDK, kThreads, kVec> tq, tk;
  Tile<T, C, kCols, kThreads, kVec> tv[kHeads];
  float gt = 0.0f;
  auto load = [&](int c) __attribute__((always_inline)) {
    const int64_t t0 = sg.begin + static_cast<int64_t>(c) * C;
    const int rows = sg.end - t0 < C ? static_cast<int>(sg.end - t0) : C;
    const int me = anew(tid);
    if (kOut) tq.load(qh + t0 * p.q.stride, p.q.stride, rows, p.q.d, me);
    tk.load(kh + t0 * p.k.stride, p.k.stride, rows, dk, me);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const T *vh = static_cast<const T *>(p.v.p) + ((h0 + i) / p.v.div) * p.v.d + j0;
      tv[i].load(vh + t0 * p.v.stride, p.v.stride, rows, dv, me);
    }
    gt = 0.0f;
    if (weighs && lane < rows) gt = decay_at(p.g, p.g_kind, t0 + lane, p.plan.heads, h);
  };
  auto stage = [&]() __attribute__((always_inline)) {
    const int me = anew(tid);
    if (kOut) tq.template store<kRowQ>(Qs, me);
    tk.template store<kRowK>(Ks, me);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) tv[i].template store<kRowV>(Vs[i], me);
    if (weighs) {
      const double a = wave_sums<C>(lane < C ? log2_decay(gt) : 0.0, lane);
      const double end = __shfl(a, C - 1);
      const float from = fast_exp2(static_cast<float>(a));
      const float to = fast_exp2(static_cast<float>(end - a));
      if (lane < C) {
        As[mine][lane] = static_cast<Sum>(a);
        Wo[mine][lane] = (kRev ? to : from) * p.inter;
        Wi[mine][lane] = (kRev ? from : to) * p.into;
      }
      if (lane == 0) Wd[mine] = fast_exp2(static_cast<float>(end));
      if (kMode == kLinState) total += end;
    }
  };

  const int first = kRev ? chunks - 1 : 0, step = kRev ? -1 : 1;
  if (chunks > 0) {
    load(first);
    stage();
  }
  for (int i = 0; i < chunks; ++i) {
    const int c = first + i * step;
    const bool more = i + 1 < chunks;
    __syncthreads();  // the chunk is staged
    if (more) load(c + step);
    Four<T, kVec> xr[kDot ? kNT : 1];  // x's rows where this lane has outputs
    if constexpr (kDot) {
      const int64_t t0 = sg.begin + static_cast<int64_t>(c) * C;
      const int rows = sg.end - t0 < C ? static_cast<int>(sg.end - t0) : C;
      const int lane = anew(tid) & 63, li = lane & 15, lq = lane >> 4;
      const T *xh = static_cast<const T *>(p.x.p) + t0 * p.x.stride + (h / p.x.div) * p.x.d + j0;
      const __amdgpu_buffer_rsrc_t v = rows_view(xh, p.x.stride, rows, dv);
      const int b = jw + 4 * lq, row = static_cast<int>(p.x.stride * sizeof(T));
      const int off = li * row + b * static_cast<int>(sizeof(T));
#pragma unroll
      for (int ti = 0; ti < kNT; ++ti) xr[ti].load(v, off + 16 * ti * row, dv - b);
    }

    __builtin_amdgcn_sched_barrier(0);
    if (kOut) {
      // token pairs: kNT x kNT tiles of 16 x 16, kSub tiles a wave of one t
      constexpr int kTiles = kNT * kNT, kBusy = kTiles < kWaves ? kTiles : kWaves;
      constexpr int kSub = kTiles / kBusy, kPer = kNT / kSub;  // waves per tile row
      const int ti = wave / kPer, s0 = wave % kPer * kSub;
      const int lane = anew(tid) & 63, li = lane & 15, lq = lane >> 4;
      if (kBusy == kWaves || wave < kBusy) {
        f32x4 acc[kSub];
#pragma unroll
        for (int si = 0; si < kSub; ++si) acc[si] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
          const Frag b = *reinterpret_cast<const Frag *>(
              &Qs[(16 * ti + li) * kRowQ + 32 * ks + 8 * lq]);
#pragma unroll
          for (int si = 0; si < kSub; ++si) {
            const Frag a = *reinterpret_cast<const Frag *>(
                &Ks[(16 * (s0 + si) + li) * kRowK + 32 * ks + 8 * lq]);
            acc[si] = mma(a, b, acc[si]);
          }
        }
        const int t = 16 * ti + li;
#pragma unroll
        for (int hd = 0; hd < kHeads; ++hd) {
          const Sum at = As[hd][t];
#pragma unroll
          for (int si = 0; si < kSub; ++si) {
            const int s = 16 * (s0 + si) + 4 * lq;
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const Sum as = As[hd][s + e];
              float w = fast_exp2(static_cast<float>(kRev ? as - at : at - as));
              asm volatile("" : "+v"(w));  // all lanes compute it: no branch for it
              x[e] = (kRev ? s + e >= t : s + e <= t) ? acc[si][e] * w * p.inside : 0.0f;
            }
            Elem *d = &Ps[hd][t * kRowP + s];
            if constexpr (kBf16)
              *reinterpret_cast<bf16x4 *>(d) = __builtin_convertvector(x, bf16x4);
            else
              *reinterpret_cast<f32x4 *>(d) = x;
          }
        }
      }
    }

    __builtin_amdgcn_sched_barrier(0);  // phases apart: their operands share registers
    f32x4 O[kNT];
    if (kOut) {
#pragma unroll
      for (int ti = 0; ti < kNT; ++ti) O[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
      // the state's part
      const int lane = anew(tid) & 63, li = lane & 15, lq = lane >> 4;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        __builtin_amdgcn_sched_barrier(0);
        const f32x8 s = __builtin_shufflevector(S[2 * ks], S[2 * ks + 1], 0, 1, 2, 3, 4, 5, 6, 7);
        const Frag hi = to_frag(s, Frag{});
        Frag mid, lo;
        if constexpr (kDot && kBf16) split(s, hi, &mid, &lo);
#pragma unroll
        for (int ti = 0; ti < kNT; ++ti) {
          const Frag b = two_halves(&Qs[(16 * ti + li) * kRowQ + 32 * ks + 4 * lq]);
          O[ti] = mma(hi, b, O[ti]);
          if constexpr (kDot && kBf16) {
            O[ti] = mma(mid, b, O[ti]);
            O[ti] = mma(lo, b, O[ti]);
          }
        }
      }
#pragma unroll
      for (int ti = 0; ti < kNT; ++ti) O[ti] *= Wo[mine][16 * ti + li];
      if constexpr (kDot) {
        // dot products of the state's part with x's rows, this wave's columns
#pragma unroll
        for (int ti = 0; ti < kNT; ++ti) {
          float d = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) d = fmaf(O[ti][e], xr[ti][e], d);
          d += __shfl_xor(d, 16);
          d += __shfl_xor(d, 32);
          if (lq == 0) Dots[wave * C + 16 * ti + li] = d;
        }
      }
    }

    if (kBeforeLast && !more && ends && p.out_seqs) save(p.out_seqs + by_seq);

    __builtin_amdgcn_sched_barrier(0);
    // into the state
    const float wd = Wd[mine];
    const int fresh = anew(tid) & 63;
#pragma unroll
    for (int it = 0; it < kIT; ++it) S[it] *= wd;
    Frag vf[kTS];
#pragma unroll
    for (int ts = 0; ts < kTS; ++ts) {
      __builtin_amdgcn_sched_barrier(0);
      const f32x8 w = two_halves(&Wi[mine][32 * ts + 4 * (fresh >> 4)]);
      vf[ts] = frag_by_column<kRowV>(Vs[mine], 32 * ts, jw, fresh);
      const f32x8 x = __builtin_convertvector(vf[ts], f32x8) * w;
      const Frag hi = to_frag(x, Frag{});
      Frag mid, lo;
      if constexpr (kBf16) split(x, hi, &mid, &lo);
#pragma unroll
      for (int it = 0; it < kIT; ++it) {
        if (it % 4 == 0) __builtin_amdgcn_sched_barrier(0);
        const Frag a = frag_by_column<kRowK>(Ks, 32 * ts, 16 * it, fresh);
        S[it] = mma(a, hi, S[it]);
        if constexpr (kBf16) {
          S[it] = mma(a, mid, S[it]);
          S[it] = mma(a, lo, S[it]);
        }
      }
    }

    __syncthreads();  // the pairs' products are in LDS; all else there is read
    if (more) stage();
    if (kOut) {
      const int lane = anew(tid) & 63, li = lane & 15, lq = lane >> 4;
      // A pair left out has the weight 0, whose product with an infinity or
      // NaN is NaN.  So columns that hold one, found by a product with zeros,
      // are cleared of them first and marked from the first one on (against
      // token order: up to the last) behind.  (1 to 3 % of a call's time; done
      // before the barrier, where more registers are in use, 9 more of them
      // went through scratch memory.)
      f32x4 none = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ts = 0; ts < kTS; ++ts) none = mma(vf[ts], Frag{}, none);
      const bool odd =
          __builtin_amdgcn_ballot_w64(!(none[0] + none[1] + none[2] + none[3] == 0.0f)) != 0;
      int mark = kRev ? -1 : C;  // of column li
      if (odd) {
#pragma unroll
        for (int ts = 0; ts < kTS; ++ts)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int s = 32 * ts + 4 * lq + e % 4 + e / 4 * 16;
            if (!(fabsf(static_cast<float>(vf[ts][e])) <= kLargest)) {
              mark = kRev ? (s > mark ? s : mark) : (s < mark ? s : mark);
              vf[ts][e] = static_cast<Elem>(0.0f);
            }
          }
#pragma unroll
        for (int d = 16; d < 64; d *= 2) {
          const int o = __shfl_xor(mark, d);
          mark = kRev ? (o > mark ? o : mark) : (o < mark ? o : mark);
        }
      }
#pragma unroll
      for (int ti = 0; ti < kNT; ++ti)
#pragma unroll
        for (int ts = 0; ts < kTS; ++ts) {
          if (kRev ? 2 * ts + 1 < ti : 2 * ts > ti) continue;  // no pair left
          const Frag b = two_halves(&Ps[mine][(16 * ti + li) * kRowP + 32 * ts + 4 * lq]);
          O[ti] = mma(vf[ts], b, O[ti]);
        }
      if (odd)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int from = __shfl(mark, 4 * lq + e);
#pragma unroll
          for (int ti = 0; ti < kNT; ++ti)
            if (kRev ? 16 * ti + li <= from : 16 * ti + li >= from) O[ti][e] = __builtin_nanf("");
        }
      const int64_t t0 = sg.begin + static_cast<int64_t>(c) * C;
      const int rows = sg.end - t0 < C ? static_cast<int>(sg.end - t0) : C;
      const int64_t out_stride = static_cast<int64_t>(p.plan.heads) * p.v.d;
      const int64_t at = t0 * out_stride + h * p.v.d + j0;
      auto write = [&](auto *out) __attribute__((always_inline)) {
        typedef std::remove_reference_t<decltype(*out)> E;
        constexpr int kSize = sizeof(E);
        const __amdgpu_buffer_rsrc_t v = rows_view(out + at, out_stride, rows, dv);
        const int b = jw + 4 * lq, row = static_cast<int>(out_stride) * kSize;
        const int off = li * row + b * kSize;
#pragma unroll
        for (int ti = 0; ti < kNT; ++ti)
          store4<kVec>(v, off + 16 * ti * row, O[ti], dv - b, E(0));
      };
      if (p.out_f32)
        write(static_cast<float *>(p.out));
      else
        write(static_cast<T *>(p.out));
      if constexpr (kDot) {
        if (tid < C && t0 + tid < sg.end) {
          float d = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) d += Dots[w * C + tid];
          p.dots[(slice * p.plan.tokens + t0 + tid) * p.plan.heads + h] = d;
        }
      }
    }
  }

  if (kMode == kLinState)
    save(p.out_slots + by_slot);
  else if (!kBeforeLast && p.out_seqs && ends)
    save(p.out_seqs + by_seq);
  if (kMode == kLinState && weighs && lane == 0 && slice == 0)
    p.out_decay[slot * p.plan.heads + h] = fast_exp2(static_cast<float>(total));
}

// -------------------------------------------------- gradient of the decay ---
// With W_ts = scale e^{a_t - a_s} (q_t . k_s) (do_t . v_s) over all pairs
// s < t of a sequence, dL/dg_t is the sum of W over the pairs that straddle
// t (s < t <= r).  From the end of a segment backwards,
//   dg_t = dg_{t+1} + (what t's row adds) - (what t's column adds),
// dg at a segment's end being the inner product of the state there with its
// adjoint.  Row and column sums leave out the pair (t, t), and pairs inside a
// chunk enter rows and columns with the same 32-bit value, so that what
// cancels, cancels: only the sums' own rounding is left.  At a sequence's
// end the adjoint (dh_final) also meets the last tokens' own terms, which no
// dg holds and which may be far larger; so the last chunk is summed from the
// state before it: dg_t = e^{a_T} <S, dh_final> + rows from t on + columns
// before t.

// Pairs inside each chunk: out_t = sum_{s<t} W_ts - sum_{r>t} W_rt, for one
// chunk of kHeads heads that share q and k.  k and v go through LDS (every
// wave needs half of their rows), q's and do's rows from memory into the
// fragments of the two waves that use them.
template <typename T, int kDKq, int kDKv, int kHeads>
struct PairsShared {
  typedef Traits<T> Tr;
  static constexpr int C = Tr::kChunk, kNT = C / 16;
  static constexpr int kSub = Tr::kBf16 ? 2 : 1, kPer = kNT / kSub;  // tiles a wave, waves a tile row
  static constexpr int kPad = Tr::kBf16 ? 16 : 4, kRowK = kDKq + kPad, kRowV = kDKv + kPad;
  alignas(16) typename Tr::Elem Ks[C * kRowK];
  alignas(16) typename Tr::Elem Vs[kHeads][C * kRowV];
  double As[kHeads][C];
  float Cols[kHeads][kNT][C];
  float Rows[kHeads][kPer][C];
};

template <typename T, int kDKq, int kDKv, int kWaves, int kHeads, bool kVec>
__device__ __forceinline__ void pairs(const LinPairs &p, unsigned block,
                                      PairsShared<T, kDKq, kDKv, kHeads> &sm) {
  typedef Traits<T> Tr;
  typedef typename Tr::Frag Frag;
  typedef PairsShared<T, kDKq, kDKv, kHeads> Shared;
  constexpr int C = Tr::kChunk, kNT = C / 16, kThreads = 64 * kWaves;
  constexpr int kSub = Shared::kSub, kPer = Shared::kPer, kBusy = kNT * kPer;
  static_assert(kBusy <= kWaves, "a wave for each part of a tile row");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const unsigned teams = static_cast<unsigned>(p.plan.heads) / kHeads;
  const int h0 = block % teams * kHeads;
  const Segment sg = segment_of(p.plan, block / teams);  // one chunk
  const int64_t t0 = sg.begin;
  if (!sg.real || t0 >= sg.end) return;
  const int rows = static_cast<int>(sg.end - t0);
  auto head = [&](const LinSide &x, int h) __attribute__((always_inline)) {
    return static_cast<const T *>(x.p) + t0 * x.stride + (h / x.div) * x.d;
  };
  const int ti = wave / kPer % kNT, s0 = wave % kPer * kSub;
  const bool some = wave < kBusy && s0 <= ti;  // else every pair of this wave's is empty
  Frag qf[kDKq / 32], of[kHeads][kDKv / 32];
  {
    Tile<T, C, kDKq, kThreads, kVec> tk;
    Tile<T, C, kDKv, kThreads, kVec> tv[kHeads];
    tk.load(head(p.k, h0), p.k.stride, rows, p.k.d, tid);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      tv[i].load(head(p.v, h0 + i), p.v.stride, rows, p.v.d, tid);
    auto rows_of = [&](const LinSide &x, int h, Frag *f, int steps) __attribute__((always_inline)) {
      const __amdgpu_buffer_rsrc_t v = rows_view(head(x, h), x.stride, rows, x.d);
#pragma unroll
      for (int ks = 0; ks < steps; ++ks) {
        const int c = 32 * ks + 8 * lq;
        f[ks] = view_frag<T, kVec>(
            v, static_cast<int>(((16 * ti + li) * x.stride + c) * sizeof(T)), some ? x.d - c : 0);
      }
    };
    rows_of(p.q, h0, qf, kDKq / 32);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) rows_of(p.o, h0 + i, of[i], kDKv / 32);
    if (wave < kHeads) {
      const float g = lane < rows ? decay_at(p.g, p.g_kind, t0 + lane, p.plan.heads, h0 + wave) : 0.0f;
      const double a = wave_sums<C>(lane < C ? log2_decay(g) : 0.0, lane);
      if (lane < C) sm.As[wave][lane] = a;
    }
    tk.template store<Shared::kRowK>(sm.Ks, tid);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) tv[i].template store<Shared::kRowV>(sm.Vs[i], tid);
  }
  __syncthreads();
  if (wave < kBusy) {
    f32x4 qk[kSub];
#pragma unroll
    for (int si = 0; si < kSub; ++si) qk[si] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (some) {
#pragma unroll
      for (int ks = 0; ks < kDKq / 32; ++ks)
#pragma unroll
        for (int si = 0; si < kSub; ++si)
          qk[si] = mma(*reinterpret_cast<const Frag *>(
                           &sm.Ks[(16 * (s0 + si) + li) * Shared::kRowK + 32 * ks + 8 * lq]),
                       qf[ks], qk[si]);
    }
    // lane: token t = 16 ti + li against s = 16 (s0 + si) + 4 lq + e
    const int t = 16 * ti + li;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const double at = sm.As[i][t];
      float row_sum = 0.0f;
#pragma unroll
      for (int si = 0; si < kSub; ++si) {
        f32x4 ov = {0.f, 0.f, 0.f, 0.f};
        if (some) {
#pragma unroll
          for (int ks = 0; ks < kDKv / 32; ++ks)
            ov = mma(*reinterpret_cast<const Frag *>(
                         &sm.Vs[i][(16 * (s0 + si) + li) * Shared::kRowV + 32 * ks + 8 * lq]),
                     of[i][ks], ov);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = 16 * (s0 + si) + 4 * lq + e;
          const float f = fast_exp2(static_cast<float>(at - sm.As[i][s])) * p.scale;
          const float x = s < t ? qk[si][e] * ov[e] * f : 0.0f;
          row_sum += x;
          float col = x;
          col += __shfl_xor(col, 1);
          col += __shfl_xor(col, 2);
          col += __shfl_xor(col, 4);
          col += __shfl_xor(col, 8);
          if (li == 0) sm.Cols[i][ti][s] = col;
        }
      }
      row_sum += __shfl_xor(row_sum, 16);
      row_sum += __shfl_xor(row_sum, 32);
      if (lq == 0) sm.Rows[i][wave % kPer][t] = row_sum;
    }
  }
  __syncthreads();
  if (tid < kHeads * C && tid % C < rows) {
    const int i = tid / C, t = tid % C;
    float c = 0.0f, r = 0.0f;
#pragma unroll
    for (int w = 0; w < kNT; ++w) c += sm.Cols[i][w][t];
#pragma unroll
    for (int w = 0; w < kPer; ++w) r += sm.Rows[i][w][t];
    p.out[(t0 + t) * p.plan.heads + h0 + i] = r - c;
  }
}

// ------------------------------------------------------------- launches ---
constexpr int waves_per_simd(int dk) { return dk > 128 ? 2 : 4; }

template <typename T, int kDK, int kWaves, int kHeads, int kMode, bool kRev, bool kVec>
__global__ __launch_bounds__(64 * kWaves, waves_per_simd(kDK)) void linattn_core_kernel(LinCore p) {
  __shared__ CoreShared<T, kDK, kWaves, kHeads, kMode> sm;
  core<T, kDK, kWaves, kHeads, kMode, kRev, kVec>(p, blockIdx.x, sm);
}

template <int kWaves, int kHeads>
unsigned core_blocks(const LinCore &a) {
  constexpr int kCols = 16 * kWaves / kHeads;
  return static_cast<unsigned>(a.plan.slots * (a.plan.heads / kHeads) *
                               ((a.v.d + kCols - 1) / kCols));
}

template <typename T, int kDK, int kWaves, int kHeads, int kMode, bool kRev>
int launch_core_t(const LinCore &a, hipStream_t s) {
  const dim3 grid(core_blocks<kWaves, kHeads>(a)), block(64 * kWaves);
  if (a.plan.vec)
    hipLaunchKernelGGL((linattn_core_kernel<T, kDK, kWaves, kHeads, kMode, kRev, true>), grid,
                       block, 0, s, a);
  else
    hipLaunchKernelGGL((linattn_core_kernel<T, kDK, kWaves, kHeads, kMode, kRev, false>), grid,
                       block, 0, s, a);
  return static_cast<int>(hipGetLastError());
}

// The class of a contracted size: what its tiles are padded to.
template <typename F>
int by_class(int d, F &&f) {
  if (d <= 64) return f(std::integral_constant<int, 64>{});
  if (d <= 128) return f(std::integral_constant<int, 128>{});
  return f(std::integral_constant<int, 256>{});
}

// Workgroups: 8 waves on 128 columns of a head; where heads have at most 64,
// on two heads that share the first two operands (which are then read, and
// multiplied, once for both); else 4 waves on 64 columns.
template <typename F>
int by_team(const LinCore &a, F &&f) {
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 2> Two;
  typedef std::integral_constant<int, 4> Four_;
  typedef std::integral_constant<int, 8> Eight;
  if (a.v.d > 64) return f(Eight{}, One{});
  if (linattn_pairs_heads(a.k.div, a.v.d)) return f(Eight{}, Two{});
  return f(Four_{}, One{});
}

// The forward output pass.
template <typename T>
int launch_out(const LinCore &a, hipStream_t s) {
  return by_class(a.k.d, [&](auto dk) {
    return by_team(a, [&](auto waves, auto heads) {
      return launch_core_t<T, dk(), waves(), heads(), kLinOut, false>(a, s);
    });
  });
}

// The states that segments add: of the forward recurrence, and with `back`
// also its adjoint's against token order, side by side in one launch.
template <typename T, int kDK, int kWaves, int kHeads, bool kVec>
__global__ __launch_bounds__(64 * kWaves, waves_per_simd(kDK)) void linattn_states_kernel(
    LinCore fwd, LinCore back, unsigned nfwd) {
  __shared__ CoreShared<T, kDK, kWaves, kHeads, kLinState> sm;
  if (blockIdx.x < nfwd)
    core<T, kDK, kWaves, kHeads, kLinState, false, kVec>(fwd, blockIdx.x, sm);
  else
    core<T, kDK, kWaves, kHeads, kLinState, true, kVec>(back, blockIdx.x - nfwd, sm);
}

template <typename T>
int launch_states(const LinCore &a, const LinCore *back, hipStream_t s) {
  return by_class(a.k.d, [&](auto dk) {
    return by_team(a, [&](auto waves, auto heads) {
      constexpr int kDK = dk(), kWaves = waves(), kHeads = heads();
      if (!back) return launch_core_t<T, kDK, kWaves, kHeads, kLinState, false>(a, s);
      const unsigned n = core_blocks<kWaves, kHeads>(a);
      const dim3 grid(2 * n), block(64 * kWaves);
      if (a.plan.vec)
        hipLaunchKernelGGL((linattn_states_kernel<T, kDK, kWaves, kHeads, true>), grid, block, 0,
                           s, a, *back, n);
      else
        hipLaunchKernelGGL((linattn_states_kernel<T, kDK, kWaves, kHeads, false>), grid, block, 0,
                           s, a, *back, n);
      return static_cast<int>(hipGetLastError());
    });
  });
}

// The three gradients and, with kDots, the sums over pairs in one launch, so
// that together they fill the GPU where one alone has too few workgroups: dq
// and dk contract over v_dim (kDKv), dv over qk_dim (kDKq).  All of one
// workgroup size; the pairs' short workgroups come last: they fill what the
// long ones leave, where the same sums inside dv's pass made it the longest of
// the three.  Measured, bf16, with the decay's gradient: 2 x 2048 tokens, 16
// heads of 128 on states of 128, 104 us (187 MB of the step's inputs and
// outputs); 4 x 2000 tokens, 24 heads of 64 on states of 128 and one q and k,
// 153 us.  Bound as the forward pass (vector issue 34 and 49 % of the time,
// waves wait 53 and 50 % of their cycles), and for heads of 128 by 16 registers
// a lane that do not fit (the dot products' rows) and go through scratch memory
// once a chunk.
template <typename T, int kDKv, int kDKq, int kWaves, int kHeads, bool kDots, bool kVec>
__global__ __launch_bounds__(64 * kWaves, waves_per_simd(kDKv > kDKq ? kDKv : kDKq)) void
linattn_grads_kernel(LinCore dq, LinCore dk, LinCore dv, LinPairs pr, unsigned n, unsigned nv) {
  constexpr int kMode = kDots ? kLinOutDot : kLinOut;
  __shared__ union {
    CoreShared<T, kDKv, kWaves, 1, kMode> a;
    CoreShared<T, kDKq, kWaves, kHeads, kLinOut> b;
    PairsShared<T, kDKq, kDKv, kHeads> c;
  } sm;
  if (blockIdx.x < nv)
    core<T, kDKq, kWaves, kHeads, kLinOut, true, kVec>(dv, blockIdx.x, sm.b);
  else if (blockIdx.x < nv + n)
    core<T, kDKv, kWaves, 1, kMode, false, kVec>(dq, blockIdx.x - nv, sm.a);
  else if (!kDots || blockIdx.x < nv + 2 * n)
    core<T, kDKv, kWaves, 1, kMode, true, kVec>(dk, blockIdx.x - nv - n, sm.a);
  else if constexpr (kDots)
    pairs<T, kDKq, kDKv, kWaves, kHeads, kVec>(pr, blockIdx.x - nv - 2 * n, sm.c);
}

template <typename T, int kDKv, int kDKq, int kWaves, int kHeads>
int launch_grads_t(const LinCore &dq, const LinCore &dk, const LinCore &dv, const LinPairs *pr,
                   hipStream_t s) {
  const unsigned n = core_blocks<kWaves, 1>(dq), nv = core_blocks<kWaves, kHeads>(dv);
  const unsigned np =
      pr ? static_cast<unsigned>(pr->plan.slots * (pr->plan.heads / kHeads)) : 0;
  const dim3 grid(2 * n + nv + np), block(64 * kWaves);
  auto go = [&](auto dots, auto vec) {
    hipLaunchKernelGGL((linattn_grads_kernel<T, kDKv, kDKq, kWaves, kHeads, dots(), vec()>), grid,
                       block, 0, s, dq, dk, dv, pr ? *pr : LinPairs{}, n, nv);
  };
  typedef std::true_type Yes;
  typedef std::false_type No;
  if (pr)
    dq.plan.vec ? go(Yes{}, Yes{}) : go(Yes{}, No{});
  else
    dq.plan.vec ? go(No{}, Yes{}) : go(No{}, No{});
  return static_cast<int>(hipGetLastError());
}

// The gradients' workgroups have 8 waves (a wave for each half row of the
// pairs' tiles); 128 columns of an output of at most 64 are then half empty,
// except where dv takes two heads.
template <typename T>
int launch_grads(const LinCore &dq, const LinCore &dk, const LinCore &dv, const LinPairs *pr,
                 hipStream_t s) {
  return by_class(dq.k.d, [&](auto cv) {
    return by_class(dv.k.d, [&](auto cq) {
      constexpr int kDKv = cv(), kDKq = cq();
      if constexpr (kDKv == 64)
        if (linattn_pairs_heads(dv.k.div, dv.v.d))
          return launch_grads_t<T, kDKv, kDKq, 8, 2>(dq, dk, dv, pr, s);
      return launch_grads_t<T, kDKv, kDKq, 8, 1>(dq, dk, dv, pr, s);
    });
  });
}

}  // namespace lin
}  // namespace ssm
