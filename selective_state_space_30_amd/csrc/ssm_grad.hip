// ssm_grad.hip -- gfx950 kernels of the gradients' global norm and clipping.
//
//   norm = sqrt(sum g^2),  g' = g min(1, max_norm / norm)
//
// Tensors are cut into chunks, which a launch's workgroups take in turn; the
// table of tensors travels in the launch's arguments.  Each workgroup adds the
// squares of its chunks in 64 bits to a sum of its own, and every workgroup of
// the clipping launch adds those sums, all in the same order, so no launch of
// one workgroup stands between the two.
#include "ssm_model_internal.h"
#include "ssm_pieces.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int kThreads = 256;

// Workgroups of the clipping launch: most take a chunk or two, for the sake of
// the last ones (with 1024, 2048, 4096, 8192 and 16384, 771 MB in fp32: 464, 462,
// 451, 443 and 443 us, 1.6 GB in bf16: 892, 888, 879, 871 and 861 us), although
// each adds the sums again.
constexpr uint32_t kScaleGroups = 16384;

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Sum over the workgroup's waves, the same in every thread.
template <int kWaves>
__device__ __forceinline__ double block_sum64(double v, double *buf) {
  v = wave_sum64(v);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) v += buf[w];
  return v;
}

// The factor of a norm, which is also rounded to what the caller is shown.  A
// norm that is infinite, NaN, or not above max_norm leaves the gradients.
__device__ __forceinline__ float factor_of(double norm, float max_norm, float &shown) {
  shown = static_cast<float>(norm);
  const double limit = static_cast<double>(max_norm);
  const bool clip = shown < __builtin_huge_valf() && norm > limit;
  return clip ? static_cast<float>(limit / norm) : 1.0f;
}

__device__ __forceinline__ double sum_of_squares(const double *sums, int n, double *buf) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v += sums[i];
  return block_sum64<kThreads / 64>(v, buf);
}

// Entry of n that has a chunk; `last`: that of the chunk before, which often has
// this one too.
__device__ __forceinline__ int entry_of(const uint32_t *first, int n, uint32_t chunk, int last) {
  if (first[last] <= chunk && chunk < first[last + 1]) return last;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *g, int n) {
  double acc[2] = {0.0, 0.0};
  int at = threadIdx.x * 8;
  auto add = [&](const Piece<T, 8> &x) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double v = static_cast<double>(x[e]);
      acc[e % 2] = fma(v, v, acc[e % 2]);
    }
  };
  for (; at + 3 * kThreads * 8 + 8 <= n; at += 4 * kThreads * 8) {
    Piece<T, 8> x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k].load(g + at + k * kThreads * 8);
#pragma unroll
    for (int k = 0; k < 4; ++k) add(x[k]);
  }
  for (; at < n; at += kThreads * 8) {
    Piece<T, 8> x;
    const int q = at / 8;
    load_piece(x, g, q, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double v = in_piece<8>(q, e, n) ? static_cast<double>(x[e]) : 0.0;
      acc[e % 2] = fma(v, v, acc[e % 2]);
    }
  }
  return acc[0] + acc[1];
}

// Bound by memory: 267 gradients of 24 layers, 771 MB in fp32, 160 us in two
// launches (4.8 TB/s; one tensor of 800 MB 5.6).  A square in 64 bits costs two
// instructions an element, a tenth of the time.
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradTable t, double *sums,
                                                               int first) {
  __shared__ double Buf[kThreads / 64];
  double acc = 0.0;
  int k = 0;
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    k = entry_of(t.first, t.n, c, k);
    const int64_t from = static_cast<int64_t>(c - t.first[k]) * kGradChunk;
    const int64_t size = static_cast<int64_t>(t.size[k] & kGradSize) - from;
    const int n = static_cast<int>(size < kGradChunk ? size : kGradChunk);
    if (t.size[k] & kGradBf16)
      acc += chunk_squares(static_cast<const uint16_t *>(t.grad[k]) + from, n);
    else
      acc += chunk_squares(static_cast<const float *>(t.grad[k]) + from, n);
  }
  acc = block_sum64<kThreads / 64>(acc, Buf);
  if (threadIdx.x == 0) sums[blockIdx.x] = first ? acc : sums[blockIdx.x] + acc;
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double *sums, int n, float *norm) {
  __shared__ double Buf[kThreads / 64];
  const double v = sum_of_squares(sums, n, Buf);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(v));
}

template <typename T, typename W>
__device__ __forceinline__ void scale_chunk(const T *g, W *out, int n, float c) {
  auto put = [&](const Piece<T, 8> &x, int at) __attribute__((always_inline)) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x[e] * c;
    store_piece<W, 8>(out, at / 8, n, v);
  };
  int at = threadIdx.x * 8;
  for (; at + 3 * kThreads * 8 + 8 <= n; at += 4 * kThreads * 8) {
    Piece<T, 8> x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k].load(g + at + k * kThreads * 8);
#pragma unroll
    for (int k = 0; k < 4; ++k) put(x[k], at + k * kThreads * 8);
  }
  for (; at < n; at += kThreads * 8) {
    Piece<T, 8> x;
    load_piece(x, g, at / 8, n);
    put(x, at);
  }
}

// Bound by memory.  The gradients above into other tensors: 276 us (1542 MB, 5.6
// TB/s), the whole call 443 us.  Taken from the end, so that what the squares'
// launch read last comes from the last-level cache: 476 -> 461 us, 1.6 GB in
// bf16 905 -> 884.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradTable t, GradOuts o, int in_place,
                                                             const double *sums, int nsums,
                                                             float max_norm, float *norm,
                                                             int write_norm) {
  __shared__ double Buf[kThreads / 64];
  const double total = sums ? sqrt(sum_of_squares(sums, nsums, Buf)) : static_cast<double>(*norm);
  float shown;
  const float c = factor_of(total, max_norm, shown);
  if (sums && write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = shown;
  if (in_place && c == 1.0f) return;
  // from the end, which was read last and may still be in the last-level cache
  int k = 0;
  for (uint32_t j = blockIdx.x; j < t.first[t.n]; j += gridDim.x) {
    const uint32_t i = t.first[t.n] - 1 - j;
    k = entry_of(t.first, t.n, i, k);
    const int64_t from = static_cast<int64_t>(i - t.first[k]) * kGradChunk;
    const int64_t size = static_cast<int64_t>(t.size[k] & kGradSize) - from;
    const int n = static_cast<int>(size < kGradChunk ? size : kGradChunk);
    const void *g = t.grad[k];
    void *out = o.out[k];
    if (t.size[k] & kGradBf16) {
      const uint16_t *x = static_cast<const uint16_t *>(g) + from;
      if (t.size[k] & kGradOutBf16)
        scale_chunk(x, static_cast<uint16_t *>(out) + from, n, c);
      else
        scale_chunk(x, static_cast<float *>(out) + from, n, c);
    } else {
      const float *x = static_cast<const float *>(g) + from;
      if (t.size[k] & kGradOutBf16)
        scale_chunk(x, static_cast<uint16_t *>(out) + from, n, c);
      else
        scale_chunk(x, static_cast<float *>(out) + from, n, c);
    }
  }
}

// All of it in one launch, for tensors of up to kGradSmall pieces of 8 elements
// together: the table counts pieces, a thread holds up to kHeld of them in
// registers between the sum and the clipping.  Eleven gradients, 32768 elements:
// 8 us, a call 10 us (with two launches 4 us more).
constexpr int kSmallThreads = 1024, kHeld = kGradSmall / kSmallThreads;
__global__ __launch_bounds__(kSmallThreads) void grad_small_kernel(GradTable t, GradOuts o,
                                                                  int clip, int in_place,
                                                                  float max_norm, float *norm) {
  __shared__ double Buf[kSmallThreads / 64];
  // the table, since each lane looks for its own entry
  __shared__ uint32_t First[kGradTensors + 1], Size[kGradTensors];
  __shared__ const void *Grad[kGradTensors];
  for (int i = threadIdx.x; i <= t.n; i += kSmallThreads) {
    First[i] = t.first[i];
    if (i == t.n) break;
    Size[i] = t.size[i];
    Grad[i] = t.grad[i];
  }
  __syncthreads();
  float v[kHeld][8];
  int entry[kHeld], q[kHeld];
  double acc = 0.0;
  const uint32_t all = First[t.n];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const uint32_t at = threadIdx.x + i * kSmallThreads;
    if (at >= all) break;
    const int k = entry_of(First, t.n, at, 0), size = Size[k] & kGradSize;
    entry[i] = k;
    q[i] = at - First[k];
    if (Size[k] & kGradBf16)
      get_piece<uint16_t, 8>(static_cast<const uint16_t *>(Grad[k]), q[i], size, v[i]);
    else
      get_piece<float, 8>(static_cast<const float *>(Grad[k]), q[i], size, v[i]);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (threadIdx.x + i * kSmallThreads >= all) break;
    const int size = Size[entry[i]] & kGradSize;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double x = in_piece<8>(q[i], e, size) ? static_cast<double>(v[i][e]) : 0.0;
      acc = fma(x, x, acc);
    }
  }
  float shown;
  const float c = factor_of(sqrt(block_sum64<kSmallThreads / 64>(acc, Buf)), max_norm, shown);
  if (threadIdx.x == 0) *norm = shown;
  if (!clip || (in_place && c == 1.0f)) return;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (threadIdx.x + i * kSmallThreads >= all) break;
    const int k = entry[i], size = Size[k] & kGradSize;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= c;
    if (Size[k] & kGradOutBf16)
      store_piece<uint16_t, 8>(static_cast<uint16_t *>(o.out[k]), q[i], size, v[i]);
    else
      store_piece<float, 8>(static_cast<float *>(o.out[k]), q[i], size, v[i]);
  }
}

}  // namespace

int launch_grad_small(const GradTable &t, const GradOuts &outs, bool clip, bool in_place,
                      float max_norm, float *norm, void *stream) {
  hipLaunchKernelGGL(grad_small_kernel, dim3(1), dim3(kSmallThreads), 0,
                     static_cast<hipStream_t>(stream), t, outs, clip ? 1 : 0, in_place ? 1 : 0,
                     max_norm, norm);
  return static_cast<int>(hipGetLastError());
}

int launch_grad_squares(const GradTable &t, double *sums, int nsums, bool first, void *stream) {
  hipLaunchKernelGGL(grad_squares_kernel, dim3(nsums), dim3(kThreads), 0,
                     static_cast<hipStream_t>(stream), t, sums, first ? 1 : 0);
  return static_cast<int>(hipGetLastError());
}

int launch_grad_norm(const double *sums, int nsums, float *norm, void *stream) {
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0,
                     static_cast<hipStream_t>(stream), sums, nsums, norm);
  return static_cast<int>(hipGetLastError());
}

int launch_grad_scale(const GradTable &t, const GradOuts &outs, bool in_place, const double *sums,
                      int nsums, float max_norm, float *norm, bool write_norm, void *stream) {
  const uint32_t chunks = t.first[t.n];
  const unsigned grid = chunks < 1 ? 1 : chunks < kScaleGroups ? chunks : kScaleGroups;
  hipLaunchKernelGGL(grad_scale_kernel, dim3(grid), dim3(kThreads), 0,
                     static_cast<hipStream_t>(stream), t, outs, in_place ? 1 : 0, sums, nsums,
                     max_norm, norm, write_norm ? 1 : 0);
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
