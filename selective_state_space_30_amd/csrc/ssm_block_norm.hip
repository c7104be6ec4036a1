// ssm_block_norm.hip -- gfx950 kernels of the block norm: the norm of a
// block's output, its gate and scale, the residual sum and the norm before
// the next block, in one pass over the rows; and its gradient in one pass.
//
// Per row, with parts of dim / groups elements:
//   u = x rsqrt(mean_part(x^2) + eps),  n = u w_post    (n = x without w_post)
//   r = residual + n silu(z) scale
//   y = r rsqrt(mean_row(r^2) + eps) w_pre
// Backward, given dr and dy, rho = rsqrt(mean(r^2) + eps):
//   D  = dr + rho (dy w_pre - r rho^2 mean(dy w_pre r))          (= dresidual)
//   dw_pre = sum_rows dy r rho,  dscale = sum_rows D n silu(z)
//   dz = D n scale silu'(z),     h = D silu(z) scale             (= dn)
//   dw_post = sum_rows h u
//   dx = s (h w_post - x s^2 mean_part(h w_post x)),  s = rsqrt(mean_part(x^2) + eps)
// n, r and u are formed again from the inputs, so the gradient is that of
// the formula and not of the rounded outputs.
//
// A workgroup takes one row at a time: every element is read once, held in
// registers in fp32, and written once; the sums over the row go through a
// wave reduction and LDS.  In the backward pass a workgroup takes every
// gridDim-th row and keeps the sums for the weights' gradients of its
// columns in registers; a second kernel adds the workgroups' sums in a fixed
// order.
#include "ssm_block_norm.h"

#include <type_traits>

#include "ssm_device.h"

namespace ssm {
namespace {

using namespace dev;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// How the sums of the parts are formed: one part (the row); parts that a
// power of two of neighbouring lanes covers; any parts (through LDS).
enum Parts { kRow = 0, kLanes = 1, kAny = 2 };

// kN neighbouring elements as they are in memory (kN = 1, or pieces of 8
// (bf16) and 4 (fp32) that are moved as a whole), and in fp32.
template <typename T, int kN>
struct Raw {
  static constexpr int kWords = kN * sizeof(T) < 4 ? 1 : kN * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kN == 1 && sizeof(T) == 2) {
      w[0] = p[0];
    } else if constexpr (kN == 1) {
      w[0] = __float_as_uint(p[0]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4 x = reinterpret_cast<const u32x4 *>(p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = x[e];
      }
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 2)
      return e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    else
      return __uint_as_float(w[e]);
  }
};
template <int kN, typename T>
__device__ __forceinline__ void get(const T *p, float (&v)[kN]) {
  Raw<T, kN> r;
  r.load(p);
#pragma unroll
  for (int e = 0; e < kN; ++e) v[e] = r[e];
}
template <int kN>
__device__ __forceinline__ void put(uint16_t *p, const float (&v)[kN]) {
  if constexpr (kN == 8) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4 *>(p) = w;
  } else {
    p[0] = from_f32<uint16_t>(v[0]);
  }
}
template <int kN>
__device__ __forceinline__ void put(float *p, const float (&v)[kN]) {
  if constexpr (kN == 1) {
    p[0] = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i)
      reinterpret_cast<f32x4 *>(p)[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Sums over the workgroup (up to 16 waves), the same in every thread.  `buf`
// may be written again once every thread has passed a later barrier, so a
// loop's calls take turns between two.
template <int kK>
__device__ __forceinline__ void block_sums(float (&v)[kK], float (*buf)[kK]) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < kK; ++k) v[k] = wave_sum(v[k]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < kK; ++k) buf[wave][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kK; ++k) v[k] = 0.0f;
  for (int w = 0; w < waves; ++w)
#pragma unroll
    for (int k = 0; k < kK; ++k) v[k] += buf[w][k];
}

// Mean over each part of the row of the products that the thread holds:
// `own` per piece in, the mean of the piece's part out.  kAny: pieces are
// single elements (kN = 1) and pass through `elems`.
template <int kParts, int kP, int kN>
__device__ __forceinline__ void part_means(float (&own)[kP], const NormArgs &p, int pieces,
                                           float (*buf)[1], float *elems, float *sums) {
  const int tid = threadIdx.x;
  const int width = p.dim / p.groups;
  const float inv = 1.0f / static_cast<float>(width);
  if constexpr (kParts == kRow) {
    float v[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kP; ++i) v[0] += own[i];
    block_sums<1>(v, buf);
#pragma unroll
    for (int i = 0; i < kP; ++i) own[i] = v[0] * inv;
  } else if constexpr (kParts == kLanes) {
    const int lanes = width / kN;
#pragma unroll
    for (int i = 0; i < kP; ++i)
      for (int d = 1; d < lanes; d *= 2) own[i] += __shfl_xor(own[i], d);
#pragma unroll
    for (int i = 0; i < kP; ++i) own[i] *= inv;
  } else {
    __syncthreads();  // the last call's readers are done
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int q = tid + i * blockDim.x;
      if (q < pieces) elems[q] = own[i];
    }
    __syncthreads();
    const int per = width / kN, waves = blockDim.x >> 6;
    for (int g = tid >> 6; g < p.groups; g += waves) {
      float s = 0.0f;
      for (int j = tid & 63; j < per; j += 64) s += elems[g * per + j];
      s = wave_sum(s);
      if ((tid & 63) == 0) sums[g] = s * inv;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int q = tid + i * blockDim.x;
      own[i] = q < pieces ? sums[q / per] : 0.0f;
    }
  }
}

// Bound by memory.  Measured: 8192 rows of 5120 bf16 in 80 parts with a gate,
// 252 MB: 41 us on inputs that the caches hold in part, 52 us a call on others
// (4.9 TB/s; a large copy: 5.2); 8192 rows of 2560 with both norms, gate, scale
// and an fp32 residual, 60 us (294 MB, 4.9 TB/s); 8 rows of 2560, 3.5 us.
template <typename T, typename R, int kN, int kP, int kParts>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormArgs p) {
  __shared__ float Buf[2][16][1];
  extern __shared__ float Dyn[];  // kAny: the row's pieces, the parts' means
  const int tid = threadIdx.x;
  const int pieces = p.dim / kN;
  float *elems = Dyn, *sums = Dyn + pieces;
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(p.x) + row * p.x_stride;
  const T *z = p.z ? static_cast<const T *>(p.z) + row * p.z_stride : nullptr;
  const R *res = p.residual ? static_cast<const R *>(p.residual) + row * p.r_stride : nullptr;
  float a[kP][kN], zz[kP][kN], rr[kP][kN];
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int q = tid + i * blockDim.x;
#pragma unroll
    for (int e = 0; e < kN; ++e) a[i][e] = zz[i][e] = rr[i][e] = 0.0f;
    if (q < pieces) {
      get<kN>(x + q * kN, a[i]);
      if (z) get<kN>(z + q * kN, zz[i]);
      if (res) get<kN>(res + q * kN, rr[i]);
    }
  }
  float s[kP];
  if (p.w_post) {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      s[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < kN; ++e) s[i] = fmaf(a[i][e], a[i][e], s[i]);
    }
    part_means<kParts, kP, kN>(s, p, pieces, Buf[0], elems, sums);
  }
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int q = tid + i * blockDim.x;
    if (q < pieces) {
      if (p.w_post) {
        const float rho = 1.0f / sqrtf(s[i] + p.eps);
        float w[kN];
        get<kN>(p.w_post + q * kN, w);
#pragma unroll
        for (int e = 0; e < kN; ++e) a[i][e] *= rho * w[e];
      }
      if (z)
#pragma unroll
        for (int e = 0; e < kN; ++e) a[i][e] *= silu_f(zz[i][e]);
      if (p.scale) {
        float w[kN];
        get<kN>(p.scale + q * kN, w);
#pragma unroll
        for (int e = 0; e < kN; ++e) a[i][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < kN; ++e) a[i][e] += rr[i][e];
      if (p.r) put<kN>(static_cast<R *>(p.r) + row * p.dim + q * kN, a[i]);
    }
  }
  if (p.y) {
    float v[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kP; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) v[0] = fmaf(a[i][e], a[i][e], v[0]);
    block_sums<1>(v, Buf[1]);
    const float rho = 1.0f / sqrtf(v[0] / static_cast<float>(p.dim) + p.eps);
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int q = tid + i * blockDim.x;
      if (q < pieces) {
        float w[kN];
        get<kN>(p.w_pre + q * kN, w);
#pragma unroll
        for (int e = 0; e < kN; ++e) w[e] *= a[i][e] * rho;
        put<kN>(static_cast<T *>(p.y) + row * p.dim + q * kN, w);
      }
    }
  }
}

// The row's inputs stay as they are in memory (packed) until they are used,
// and the next row's are asked for before this row's sums.  Measured: 8192
// rows of 2560, both norms, gate, scale, fp32 residual, 134 us on inputs that
// the caches do not hold (462 MB, 3.4 TB/s), 126 us on others (175 us without
// the early loads).  The sums for the weights leave room for one workgroup a
// CU, whose 5 waves on 4 SIMDs issue vector instructions 36 % of the time (58 %
// on the SIMD with two) and wait 46 % of their cycles.  (With those sums in LDS,
// two a CU: 181 to 211 us.)  1001 rows of 1537 in fp32, both norms and scale: 27
// us; a row a workgroup, so that 18 of the 31 MB written are partial sums.
template <typename T, typename R, int kN, int kP, int kParts, int kBound>
__global__ __launch_bounds__(kBound, sizeof(R) == 2 && kN == 8 ? 3 : 1) void norm_bwd_kernel(NormArgs p) {
  __shared__ float Buf1[16][1];
  __shared__ float Buf2[4][16][2];
  extern __shared__ float Dyn[];
  const int tid = threadIdx.x;
  const int pieces = p.dim / kN;
  float *elems = Dyn, *sums = Dyn + pieces;
  float wpost[kP][kN], wscale[kP][kN], wpre[kP][kN];
  float gpost[kP][kN], gscale[kP][kN], gpre[kP][kN];
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int q = tid + i * blockDim.x;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      wpost[i][e] = wscale[i][e] = 1.0f;
      wpre[i][e] = gpost[i][e] = gscale[i][e] = gpre[i][e] = 0.0f;
    }
    if (q < pieces) {
      if (p.w_post) get<kN>(p.w_post + q * kN, wpost[i]);
      if (p.scale) get<kN>(p.scale + q * kN, wscale[i]);
      if (p.w_pre) get<kN>(p.w_pre + q * kN, wpre[i]);
    }
  }
  // a row's inputs as they are in memory: the next row's are asked for while
  // this one's are worked on
  Raw<T, kN> rx[kP], rz[kP], ry[kP];
  Raw<R, kN> rres[kP], rdr[kP];
  auto load = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int q = tid + i * blockDim.x;
      if (q < pieces) {
        rx[i].load(static_cast<const T *>(p.x) + row * p.x_stride + q * kN);
        if (p.z) rz[i].load(static_cast<const T *>(p.z) + row * p.z_stride + q * kN);
        if (p.residual)
          rres[i].load(static_cast<const R *>(p.residual) + row * p.r_stride + q * kN);
        if (p.dy) ry[i].load(static_cast<const T *>(p.dy) + row * p.dim + q * kN);
        if (p.dr) rdr[i].load(static_cast<const R *>(p.dr) + row * p.dim + q * kN);
      }
    }
  };
  auto squares = [&](float (&s)[kP]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      s[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < kN; ++e) s[i] = fmaf(rx[i][e], rx[i][e], s[i]);
    }
  };
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    rx[i].zero();
    rz[i].zero();
    rres[i].zero();
    ry[i].zero();
    rdr[i].zero();
  }
  float s[kP];  // x's means of squares, of this row and, at its end, of the next
  load(blockIdx.x);
  if (p.w_post) {
    squares(s);
    part_means<kParts, kP, kN>(s, p, pieces, Buf1, elems, sums);
  }
  int turn = 0;  // of the buffers: a row's sums may not meet the last row's readers
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    // x, z and dy stay as they are in memory (16-bit ones take half the registers)
    Raw<T, kN> cx[kP], cz[kP], cy[kP];
    float rr[kP][kN], dd[kP][kN];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      s[i] = p.w_post ? 1.0f / sqrtf(s[i] + p.eps) : 1.0f;
      cx[i] = rx[i];
      cz[i] = rz[i];
      cy[i] = ry[i];
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        rr[i][e] = rres[i][e];
        dd[i][e] = rdr[i][e];
      }
    }
    const bool more = row + gridDim.x < p.rows;
    if (more) load(row + gridDim.x);
    // r in rr
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kP; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const float g = p.z ? silu_f(cz[i][e]) : 1.0f;
        rr[i][e] = fmaf(cx[i][e] * s[i] * wpost[i][e] * g, wscale[i][e], rr[i][e]);
        v[0] = fmaf(rr[i][e], rr[i][e], v[0]);
        v[1] = fmaf(cy[i][e] * wpre[i][e], rr[i][e], v[1]);
      }
    if (p.dy) {
      block_sums<2>(v, Buf2[turn]);
      const float rho = 1.0f / sqrtf(v[0] / static_cast<float>(p.dim) + p.eps);
      const float m = v[1] / static_cast<float>(p.dim) * rho * rho;
#pragma unroll
      for (int i = 0; i < kP; ++i) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          gpre[i][e] = fmaf(cy[i][e] * rho, rr[i][e], gpre[i][e]);
          dd[i][e] = fmaf(rho, fmaf(-m, rr[i][e], cy[i][e] * wpre[i][e]), dd[i][e]);
        }
      }
    }
    // dd: the gradient of r.  rr becomes h w_post
    float t[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int q = tid + i * blockDim.x;
      t[i] = 0.0f;
      if (q < pieces && p.dresidual)
        put<kN>(static_cast<R *>(p.dresidual) + row * p.dim + q * kN, dd[i]);
      float dz[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        // silu(z) = z sg, its slope sg (1 + z (1 - sg))
        const float z = cz[i][e], sg = sigmoid_f(z);
        const float g = p.z ? z * sg : 1.0f;
        const float u = cx[i][e] * s[i], n = u * wpost[i][e];
        gscale[i][e] = fmaf(dd[i][e], n * g, gscale[i][e]);
        dz[e] = dd[i][e] * n * wscale[i][e] * sg * fmaf(z, 1.0f - sg, 1.0f);
        const float h = dd[i][e] * g * wscale[i][e];
        gpost[i][e] = fmaf(h, u, gpost[i][e]);
        rr[i][e] = h * wpost[i][e];
        t[i] = fmaf(rr[i][e], cx[i][e], t[i]);
      }
      if (q < pieces && p.dz) put<kN>(static_cast<T *>(p.dz) + row * p.dim + q * kN, dz);
    }
    float next[kP];
    if (p.w_post) {
      // the mean of this row's h w_post x, and of the next row's x^2, by one
      // reduction where the part is the row
      if (more) squares(next);
      if constexpr (kParts == kRow) {
        float w[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          w[0] += t[i];
          w[1] += more ? next[i] : 0.0f;
        }
        block_sums<2>(w, Buf2[2 + turn]);
        const float inv = 1.0f / static_cast<float>(p.dim);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          t[i] = w[0] * inv;
          next[i] = w[1] * inv;
        }
      } else {
        part_means<kParts, kP, kN>(t, p, pieces, Buf1, elems, sums);
        if (more) part_means<kParts, kP, kN>(next, p, pieces, Buf1, elems, sums);
      }
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int q = tid + i * blockDim.x;
      if (q < pieces) {
        if (p.w_post) {
          const float m = t[i] * s[i] * s[i];
#pragma unroll
          for (int e = 0; e < kN; ++e) rr[i][e] = s[i] * fmaf(-m, cx[i][e], rr[i][e]);
        }
        put<kN>(static_cast<T *>(p.dx) + row * p.dim + q * kN, rr[i]);
      }
      s[i] = next[i];
    }
    turn ^= 1;
  }
  float *part = p.parts + static_cast<int64_t>(blockIdx.x) * 3 * p.dim;
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int q = tid + i * blockDim.x;
    if (q < pieces) {
      if (p.dw_post) put<kN>(part + q * kN, gpost[i]);
      if (p.dscale) put<kN>(part + p.dim + q * kN, gscale[i]);
      if (p.dw_pre) put<kN>(part + 2 * p.dim + q * kN, gpre[i]);
    }
  }
}

// Sum of the workgroups' partial rows, 32 columns and 32 row groups a
// workgroup, in a fixed order.  (8 us for 3 x 2560 columns.)
__global__ __launch_bounds__(1024) void norm_parts_kernel(NormArgs p) {
  __shared__ float Sums[32][33];
  const int tid = threadIdx.x, lane = tid & 31, grp = tid >> 5;
  const int which = blockIdx.y;
  float *out = which == 0 ? p.dw_post : which == 1 ? p.dscale : p.dw_pre;
  if (!out) return;
  const int c = blockIdx.x * 32 + lane;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < p.dim) {
    const float *s = p.parts + static_cast<int64_t>(which) * p.dim + c;
    const int64_t row = 3 * static_cast<int64_t>(p.dim);
    int w = grp;
    for (; w + 96 < p.nparts; w += 128)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += s[(w + 32 * k) * row];
    for (; w < p.nparts; w += 32) acc[0] += s[w * row];
  }
  Sums[grp][lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  __syncthreads();
  if (grp == 0 && c < p.dim) {
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < 32; ++g) s += Sums[g][lane];
    out[c] = s;
  }
}

// Pieces a thread holds (1, 2, 4, 8 or 16) and threads of a workgroup: whole
// pieces one each up to 1024 threads, single elements up to 512 threads, then
// more each.
struct Shape {
  int per, threads;
};
Shape shape_of(int dim, int n) {
  const int pieces = dim / n;
  const int most_per = n > 1 ? 4 : 16;
  int per = 1;
  while (per < most_per && pieces > per * (n > 1 ? 1024 : 512)) per *= 2;
  return {per, ((pieces + per - 1) / per + 63) / 64 * 64};
}

int piece_of(bool bf16, bool vec) { return vec ? (bf16 ? 8 : 4) : 1; }

template <typename T, typename R, int kN, int kP, bool kBack>
int launch_norm_p(const NormArgs &a, int threads, hipStream_t s) {
  const int width = a.dim / a.groups, lanes = width / kN;
  const bool neighbours =
      width % kN == 0 && lanes <= 64 && (lanes & (lanes - 1)) == 0 && lanes > 0;
  const int parts = !a.w_post || a.groups == 1 ? kRow : neighbours ? kLanes : kAny;
  const unsigned grid = static_cast<unsigned>(kBack ? a.nparts : a.rows);
  const size_t dyn = parts == kAny ? (a.dim / kN + a.groups) * sizeof(float) : 0;
  auto go = [&](auto kind) {
    constexpr int kKind = decltype(kind)::value;
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), dyn, s, a);
      return static_cast<int>(hipGetLastError());
    };
    if constexpr (!kBack) {
      return run(norm_fwd_kernel<T, R, kN, kP, kKind>);
    } else {
      // it holds up to 190 values a thread: 256, 168 or 128 registers
      return threads <= 512   ? run(norm_bwd_kernel<T, R, kN, kP, kKind, 512>)
             : threads <= 768 ? run(norm_bwd_kernel<T, R, kN, kP, kKind, 768>)
                              : run(norm_bwd_kernel<T, R, kN, kP, kKind, 1024>);
    }
  };
  if (parts == kRow) return go(std::integral_constant<int, kRow>{});
  if (parts == kLanes) return go(std::integral_constant<int, kLanes>{});
  return go(std::integral_constant<int, kAny>{});
}

template <typename T, typename R, int kN, bool kBack>
int launch_norm_n(const NormArgs &a, hipStream_t s) {
  const Shape sh = shape_of(a.dim, kN);
  if (sh.per == 1) return launch_norm_p<T, R, kN, 1, kBack>(a, sh.threads, s);
  if (sh.per == 2) return launch_norm_p<T, R, kN, 2, kBack>(a, sh.threads, s);
  if (sh.per == 4) return launch_norm_p<T, R, kN, 4, kBack>(a, sh.threads, s);
  if constexpr (kN == 1) {
    if (sh.per == 8) return launch_norm_p<T, R, kN, 8, kBack>(a, sh.threads, s);
    return launch_norm_p<T, R, kN, 16, kBack>(a, sh.threads, s);
  }
  return static_cast<int>(hipErrorInvalidValue);
}

template <typename T, typename R>
int launch_norm_1(const NormArgs &a, bool backward, hipStream_t s) {
  return backward ? launch_norm_n<T, R, 1, true>(a, s) : launch_norm_n<T, R, 1, false>(a, s);
}

int launch_norm(const NormArgs &a, bool backward, bool bf16, hipStream_t s) {
  // whole pieces only where no part ends inside one
  const int n = piece_of(bf16, a.vec && (a.dim / a.groups) % (bf16 ? 8 : 4) == 0);
  if (bf16) {
    if (a.wide)
      return n > 1 ? (backward ? launch_norm_n<uint16_t, float, 8, true>(a, s)
                               : launch_norm_n<uint16_t, float, 8, false>(a, s))
                   : launch_norm_1<uint16_t, float>(a, backward, s);
    return n > 1 ? (backward ? launch_norm_n<uint16_t, uint16_t, 8, true>(a, s)
                             : launch_norm_n<uint16_t, uint16_t, 8, false>(a, s))
                 : launch_norm_1<uint16_t, uint16_t>(a, backward, s);
  }
  return n > 1 ? (backward ? launch_norm_n<float, float, 4, true>(a, s)
                           : launch_norm_n<float, float, 4, false>(a, s))
               : launch_norm_1<float, float>(a, backward, s);
}

}  // namespace

int norm_parts(int64_t rows) {
  return static_cast<int>(rows < kNormMaxParts ? rows : kNormMaxParts);
}

int launch_block_norm_fwd(const NormArgs &a, bool bf16, void *stream) {
  return launch_norm(a, false, bf16, static_cast<hipStream_t>(stream));
}

int launch_block_norm_bwd(const NormArgs &a, bool bf16, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int err = a.rows > 0 ? launch_norm(a, true, bf16, s) : 0;
  if (err != 0 || (!a.dw_post && !a.dscale && !a.dw_pre)) return err;
  hipLaunchKernelGGL(norm_parts_kernel, dim3(static_cast<unsigned>((a.dim + 31) / 32), 3),
                     dim3(1024), 0, s, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
