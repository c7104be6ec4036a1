// ssm_layer_norm.hip -- gfx950 kernels of the layer norm with the residual sum
// before it, and of its gradient.
//
// Per row of dim elements:
//   r = x + residual,  m = mean(r),  s = 1 / sqrt(mean((r - m)^2) + eps)
//   y = (r - m) s weight + bias
// Backward, with h = (r - m) s and g = dy weight:
//   D = dr + s (g - mean(g) - h mean(g h))      (= dx = dresidual)
//   dweight = sum_rows dy h,  dbias = sum_rows dy
//
// The row is held in registers in fp32 by a group of lanes, kP pieces of kN
// elements each: 8 to 64 lanes of a wave, whose sums need no barrier, or a
// workgroup of up to 8 waves, whose sums meet in LDS.  The mean is formed
// first and the squares from the differences, so that a mean far from 0 costs
// only the digits that fp32 does not hold beside it.
#include "ssm_model_internal.h"
#include "ssm_pieces.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int kCus = 256;

// Sums of v over the group, the same in every lane.  `lanes` over 64: the
// workgroup.  `turn` is another one of the buffers at each call, of which two
// calls in a row have different ones: a wave writes again only behind a
// barrier that the readers have passed.
template <int kK>
__device__ __forceinline__ void row_sums(float (&v)[kK], int lanes, float (*buf)[8][2], int &turn) {
#pragma unroll
  for (int k = 0; k < kK; ++k) v[k] = group_sum(v[k], lanes);
  if (lanes <= 64) return;
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < kK; ++k) buf[turn][wave][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kK; ++k) v[k] = 0.0f;
  for (int w = 0; w < waves; ++w)
#pragma unroll
    for (int k = 0; k < kK; ++k) v[k] += buf[turn][w][k];
  turn ^= 1;
}

// The row fills every lane's pieces (kWhole), or all but the last of each.
// Whether element e of a lane's piece i lies in the row:
template <bool kWhole, int kP, int kN>
__device__ __forceinline__ bool inside(const LayerNormArgs &p, int lanes, int at, int i, int e) {
  return kWhole || i < kP - 1 || in_piece<kN>(at + i * lanes, e, p.dim);
}
template <typename T, int kN>
__device__ __forceinline__ void load_at(bool whole, Piece<T, kN> &x, const T *row, int q, int dim) {
  if (whole) {
    x.load(row + q * kN);
  } else {
    x.zero();
    if (q * kN < dim) load_piece(x, row, q, dim);
  }
}
template <typename T, int kN>
__device__ __forceinline__ void store_at(bool whole, T *row, int q, int dim, const float (&v)[kN]) {
  if (whole) {
    Piece<T, kN> x;
    x.set(v);
    x.store(row + q * kN);
  } else {
    if (q * kN < dim) store_piece<T, kN>(row, q, dim, v);
  }
}

// r - mean in v (0 behind the row's end), and s.  The mean of the differences,
// which is what the first mean's rounding left, is taken from both.  In a row of
// one value nothing else is left, and the difference of two equal sums that is the
// variance comes out as their roundings, below 0 as well (up to 42 additions each,
// 2^-24 an addition).  It is held at 2^-20 of the first sum, which is not more than
// they can round by, but is positive and leaves (the differences round to 42 *
// 2^-24 of what was taken from them) at most 42 * 2^-14 of any such row.  It matters
// where a row spreads by less than 2^-10 of what the first mean was off by, which
// is less than 42 * 2^-34 of that mean.  (A third sum,
// over the differences of the differences, cost the backward pass 10 % at rows of
// 2560 in bf16 and 19 % at rows of 8192: its registers.)
template <int kP, int kN, bool kWhole>
__device__ __forceinline__ float centre(float (&v)[kP][kN], const LayerNormArgs &p, int lanes,
                                        int at, float (*buf)[8][2], int &turn) {
  const float n = static_cast<float>(p.dim);
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < kP; ++i)
#pragma unroll
    for (int e = 0; e < kN; ++e)
      s[0] += inside<kWhole, kP, kN>(p, lanes, at, i, e) ? v[i][e] : 0.0f;
  row_sums<1>(s, lanes, buf, turn);
  const float mean = s[0] / n;
  float t[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kP; ++i)
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      v[i][e] = inside<kWhole, kP, kN>(p, lanes, at, i, e) ? v[i][e] - mean : 0.0f;
      t[0] += v[i][e];
      t[1] = fmaf(v[i][e], v[i][e], t[1]);
    }
  row_sums<2>(t, lanes, buf, turn);
  const float rest = t[0] / n;
#pragma unroll
  for (int i = 0; i < kP; ++i)
#pragma unroll
    for (int e = 0; e < kN; ++e)
      v[i][e] = inside<kWhole, kP, kN>(p, lanes, at, i, e) ? v[i][e] - rest : 0.0f;
  const float square = t[1] / n;
  return 1.0f / sqrtf(fmaxf(fmaf(-rest, rest, square), 0x1p-20f * square) + p.eps);
}

// Bound by memory, the weights in registers over the group's rows.  16384 rows
// of 2560, bf16 with an fp32 residual, 97 us (503 MB, 5.2 TB/s, as a large
// copy); 65536 of 768, all bf16, 66 us in a training step (403 MB, 6.1 TB/s: some of
// it is in the last-level cache; 75 us by itself).  With the weights read for each
// row the first took 113 us.  8 rows of 2560: 4 us, a call 9.3 us on the host.
template <typename T, typename R, typename Y, int kN, int kP, bool kWhole>
__global__ __launch_bounds__(512) void layer_norm_fwd_kernel(LayerNormArgs p, int lanes) {
  __shared__ float Buf[2][8][2];
  int turn = 0;
  const int at = threadIdx.x & (lanes - 1);
  const int per = blockDim.x / lanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int64_t row = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / lanes;
  Piece<float, kN> w[kP], b[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int q = at + i * lanes;
    if (p.weight) load_at(kWhole || i < kP - 1, w[i], p.weight, q, p.dim);
    if (p.bias) load_at(kWhole || i < kP - 1, b[i], p.bias, q, p.dim);
  }
  for (; row < p.rows; row += step) {
    float v[kP][kN];
    {
      Piece<T, kN> x[kP];
#pragma unroll
      for (int i = 0; i < kP; ++i)
        load_at(kWhole || i < kP - 1, x[i], static_cast<const T *>(p.x) + row * p.x_stride, at + i * lanes, p.dim);
      if (p.residual) {
        Piece<R, kN> res[kP];
#pragma unroll
        for (int i = 0; i < kP; ++i)
          load_at(kWhole || i < kP - 1, res[i], static_cast<const R *>(p.residual) + row * p.r_stride,
                          at + i * lanes, p.dim);
#pragma unroll
        for (int i = 0; i < kP; ++i)
#pragma unroll
          for (int e = 0; e < kN; ++e) v[i][e] = x[i][e] + res[i][e];
      } else {
#pragma unroll
        for (int i = 0; i < kP; ++i)
#pragma unroll
          for (int e = 0; e < kN; ++e) v[i][e] = x[i][e];
      }
    }
    if (p.r)
#pragma unroll
      for (int i = 0; i < kP; ++i)
        store_at<R, kN>(kWhole || i < kP - 1, static_cast<R *>(p.r) + row * p.dim, at + i * lanes, p.dim, v[i]);
    const float s = centre<kP, kN, kWhole>(v, p, lanes, at, Buf, turn);
#pragma unroll
    for (int i = 0; i < kP; ++i) {
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        v[i][e] *= s;
        if (p.weight) v[i][e] *= w[i][e];
        if (p.bias) v[i][e] += b[i][e];
      }
      store_at<Y, kN>(kWhole || i < kP - 1, static_cast<Y *>(p.y) + row * p.dim, at + i * lanes, p.dim, v[i]);
    }
  }
}

// The weight, in LDS by pieces' quarters so that neighbouring lanes read
// neighbouring 16 bytes.
template <bool kWhole, int kN>
__device__ __forceinline__ void stage_weight(const LayerNormArgs &p, float *W, int pieces) {
  for (int j = threadIdx.x; j < pieces * kN; j += blockDim.x) {
    const int q = j / kN, e = j % kN;
    const int c = kWhole || (q + 1) * kN <= p.dim ? j : p.dim - kN + e;
    const bool in = kWhole || (q * kN < p.dim && in_piece<kN>(q, e, p.dim));
    W[((e / 4) * pieces + q) * 4 + e % 4] = in ? (p.weight ? p.weight[c] : 1.0f) : 0.0f;
  }
  __syncthreads();
}

// The sums for the weights' gradients of a lane's columns stay in registers
// over the rows that its group takes; at the end the workgroup's groups are
// added in LDS in a fixed order and leave one partial row.  The weight is read
// from LDS for each row: in registers it does not fit beside them.  8192 rows of
// 2560, bf16 with an fp32 residual, 83 us (377 MB, 4.6 TB/s; 107 us without the
// next row asked for ahead, 143 us with the weight in registers, which spilled);
// vector instructions are issued 42 % of the time.  65536 of 768, all bf16, 118
// us in a training step (503 MB, 4.3 TB/s; 106 us by itself).  Rows over 8192 elements find no registers for the next
// row, nor in part for their own: 2048 of 16384, bf16, 111 us (336 MB, 3.0 TB/s;
// with 1024 threads, which spill more, the same).
template <typename T, typename R, typename Y, int kN, int kP, bool kWhole, int kBound>
__global__ __launch_bounds__(kBound) void layer_norm_bwd_kernel(LayerNormArgs p, int lanes) {
  __shared__ float Buf[2][8][2];
  extern __shared__ float Dyn[];  // the weight; at the end the groups' sums
  int turn = 0;
  const int at = threadIdx.x & (lanes - 1);
  const int per = blockDim.x / lanes;
  const int pieces = kP * lanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  const float n = static_cast<float>(p.dim);
  float gw[kP][kN], gb[kP][kN];
#pragma unroll
  for (int i = 0; i < kP; ++i)
#pragma unroll
    for (int e = 0; e < kN; ++e) gw[i][e] = gb[i][e] = 0.0f;
  auto weight = [&](int i, float (&w)[kN]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < kN / 4; ++h) {
      const float4 x = reinterpret_cast<const float4 *>(Dyn)[h * pieces + at + i * lanes];
      w[4 * h] = x.x;
      w[4 * h + 1] = x.y;
      w[4 * h + 2] = x.z;
      w[4 * h + 3] = x.w;
    }
  };
  // a row's inputs as they are in memory: the next row's are asked for before
  // this one's are worked on, unless 8 waves share the registers
  constexpr bool kAhead = kBound <= 256 || kP * kN <= 16;
  Piece<T, kN> nx[kP];
  Piece<R, kN> nres[kP], ndr[kP];
  Piece<Y, kN> ndy[kP];
  auto load = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int q = at + i * lanes;
      load_at(kWhole || i < kP - 1, nx[i], static_cast<const T *>(p.x) + row * p.x_stride, q, p.dim);
      if (p.residual)
        load_at(kWhole || i < kP - 1, nres[i], static_cast<const R *>(p.residual) + row * p.r_stride, q, p.dim);
      load_at(kWhole || i < kP - 1, ndy[i], static_cast<const Y *>(p.dy) + row * p.dim, q, p.dim);
      if (p.dr) load_at(kWhole || i < kP - 1, ndr[i], static_cast<const R *>(p.dr) + row * p.dim, q, p.dim);
    }
  };
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    nres[i].zero();
    ndr[i].zero();
  }
  int64_t row = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / lanes;
  if (kAhead && row < p.rows) load(row);
  stage_weight<kWhole, kN>(p, Dyn, pieces);
  for (; row < p.rows; row += step) {
    if (!kAhead) load(row);
    float v[kP][kN];
    Piece<Y, kN> dy[kP];
    Piece<R, kN> dr[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      dy[i] = ndy[i];
      dr[i] = ndr[i];
#pragma unroll
      for (int e = 0; e < kN; ++e) v[i][e] = nx[i][e] + nres[i][e];
    }
    if (kAhead && row + step < p.rows) load(row + step);
    const float s = centre<kP, kN, kWhole>(v, p, lanes, at, Buf, turn);
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      float w[kN];
      weight(i, w);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        v[i][e] *= s;
        const float d = inside<kWhole, kP, kN>(p, lanes, at, i, e) ? dy[i][e] : 0.0f;
        const float g = d * w[e];
        gb[i][e] += d;
        gw[i][e] = fmaf(d, v[i][e], gw[i][e]);
        m[0] += g;
        m[1] = fmaf(g, v[i][e], m[1]);
      }
    }
    row_sums<2>(m, lanes, Buf, turn);
    m[0] /= n;
    m[1] /= n;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      float w[kN], d[kN];
      weight(i, w);
#pragma unroll
      for (int e = 0; e < kN; ++e)
        d[e] = fmaf(s, fmaf(-m[1], v[i][e], fmaf(dy[i][e], w[e], -m[0])), dr[i][e]);
      store_at<T, kN>(kWhole || i < kP - 1, static_cast<T *>(p.dx) + row * p.dim, at + i * lanes, p.dim, d);
      if (p.dresidual)
        store_at<R, kN>(kWhole || i < kP - 1, static_cast<R *>(p.dresidual) + row * p.dim, at + i * lanes, p.dim, d);
    }
  }
  if (!p.dweight && !p.dbias) return;
  float *part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
  if (per > 1) {
    // groups inside a wave, then the waves one after another
#pragma unroll
    for (int i = 0; i < kP; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e)
        for (int d = lanes; d < 64; d *= 2) {
          gw[i][e] += __shfl_xor(gw[i][e], d);
          gb[i][e] += __shfl_xor(gb[i][e], d);
        }
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    __syncthreads();  // the weight is read
    for (int k = 0; k < waves; ++k) {
      if (wave == k && lane < lanes)
#pragma unroll
        for (int i = 0; i < kP; ++i)
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            float *c = Dyn + (i * kN + e) * 64 + lane;
            if (k > 0) {
              gw[i][e] += c[0];
              gb[i][e] += c[kN * kP * 64];
            }
            c[0] = gw[i][e];
            c[kN * kP * 64] = gb[i][e];
          }
      __syncthreads();
    }
    if (wave != waves - 1 || lane >= lanes) return;
  }
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    store_at<float, kN>(kWhole || i < kP - 1, part, at + i * lanes, p.dim, gw[i]);
    store_at<float, kN>(kWhole || i < kP - 1, part + p.dim, at + i * lanes, p.dim, gb[i]);
  }
}

// Sum of the workgroups' partial rows, 32 columns and 32 row groups a
// workgroup, in a fixed order.  (5 us for 2 x 2560 columns of 512 rows.)
__global__ __launch_bounds__(1024) void layer_norm_parts_kernel(LayerNormArgs p) {
  __shared__ float Sums[32][33];
  const int tid = threadIdx.x, lane = tid & 31, grp = tid >> 5;
  float *out = blockIdx.y == 0 ? p.dweight : p.dbias;
  if (!out) return;
  const int c = blockIdx.x * 32 + lane;
  constexpr int kAhead = 8;
  float acc = 0.0f;
  if (c < p.dim) {
    const float *s = p.parts + static_cast<int64_t>(blockIdx.y) * p.dim + c;
    const int64_t row = 2 * static_cast<int64_t>(p.dim);
    for (int w = grp; w < p.nparts; w += 32 * kAhead) {
      float v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v[k] = s[(w + 32 * k < p.nparts ? w + 32 * k : w) * row];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) acc += w + 32 * k < p.nparts ? v[k] : 0.0f;
    }
  }
  Sums[grp][lane] = acc;
  __syncthreads();
  if (grp == 0 && c < p.dim) {
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < 32; ++g) s += Sums[g][lane];
    out[c] = s;
  }
}

// Lanes of a row's group (a power of two, 8..512), pieces that each holds, and
// whether they fill the row.
struct Shape {
  int lanes, per, threads;
  bool whole;
};

// One wave or a part of it where its lanes hold the row in at most `alone`
// pieces each (no barrier), else as many waves as leave `shared` pieces.  Among
// up to 64 lanes the most that fill the row, since short rows want many lanes
// (forward pass, bf16: 100000 x 256 with 8, 16 and 32 lanes 43, 40 and 39 us)
// and filled ones no checks (65536 x 768 with 32 filled lanes 75 us, with 64
// not filled 78).  Long rows want fewer pieces a lane than the registers hold
// (forward, bf16: 8192 x 5120 with 128 and 256 lanes 77 and 65 us, 4096 x 8192
// with 256 and 512 lanes 57 and 52 us; backward: 8192 x 4096 with 128 and 256
// lanes 85 and 78 us, 8192 x 2560 with an fp32 residual with 64, 128 and 256
// lanes 86, 87 and 82 us).  The limits of fp32 rows (pieces of 4) are about the same
// elements a lane, and were held against others at one size only (2003 x 1537,
// backward, with 1 to 4 pieces 24 to 28 us, with 7 24 us).
Shape shape_of(int dim, int n, int alone, int shared) {
  const int pieces = (dim + n - 1) / n;
  auto per = [&](int lanes) { return (pieces + lanes - 1) / lanes; };
  int lanes = 0;
  for (int k = 64; k >= 8; k /= 2)
    if (!lanes && pieces % k == 0 && dim % n == 0 && per(k) <= alone) lanes = k;
  if (!lanes) {
    lanes = 8;
    while (lanes < 64 && per(lanes) > 1) lanes *= 2;
    if (per(lanes) > alone)
      while (lanes < 512 && per(lanes) > shared) lanes *= 2;
  }
  return {lanes, per(lanes), lanes <= 64 ? 256 : lanes, per(lanes) * lanes * n == dim};
}

// types: of elements per piece n, and whether rows are read as fp32 beside bf16
Shape shape_of(int dim, LayerNormTypes types, bool backward) {
  if (types == kLnF32) return backward ? shape_of(dim, 4, 7, 5) : shape_of(dim, 4, 8, 6);
  return shape_of(dim, 8, 4, backward && types != kLnBf16 ? 2 : 3);
}

// Workgroups that take the rows, at most `most`.
int groups_of(int64_t rows, const Shape &sh, int most) {
  const int per = sh.threads / sh.lanes;
  const int64_t groups = (rows + per - 1) / per;
  return static_cast<int>(groups < most ? groups : most);
}

// Of the forward pass: what 4 waves a SIMD make (twice as many workgroups of 512
// threads: 4096 x 8192 in bf16 53 instead of 51 us).
int forward_groups(int64_t rows, const Shape &sh) {
  return groups_of(rows, sh, kCus * 1024 / sh.threads);
}

// Workgroups a CU of the backward pass: one that asks for its rows ahead keeps
// the memory busy by itself where its lanes are filled and wait for no other
// wave; two where they fit into the registers and it does not.  (bf16, one and
// two: 32768 x 1024 69 and 73 us, 65536 x 768 105 and 109; 8192 x 4096 94 and
// 78, 30000 x 1100 95 and 76, 8192 x 2560 76 and 58; with an fp32 residual 8192
// x 2560 103 and 83.  fp32 rows take the limit of those with an fp32 residual,
// not measured by themselves.)
int back_groups(int64_t rows, const Shape &sh, LayerNormTypes types) {
  const int held = sh.per * (types == kLnF32 ? 4 : 8);
  const bool fit = held <= (types == kLnBf16 ? 24 : 16) && sh.threads <= 256;
  const int each = fit && (!sh.whole || sh.lanes > 64) ? 2 : 1;
  return groups_of(rows, sh, each * kCus * 256 / (sh.threads < 256 ? sh.threads : 256));
}

template <typename T, typename R, typename Y, int kN, int kP, bool kWhole, bool kBack>
int launch_p(const LayerNormArgs &a, const Shape &sh, hipStream_t s) {
  if constexpr (kBack) {
    const size_t weight = static_cast<size_t>(kN) * kP * sh.lanes * 4;
    const size_t sums = sh.lanes <= 64 ? 2 * kN * kP * 64 * 4 : 0;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(a.nparts), dim3(sh.threads), weight > sums ? weight : sums, s,
                         a, sh.lanes);
      return static_cast<int>(hipGetLastError());
    };
    // 512 lanes take what 256 hold in no `shared` pieces each (5 of 4 elements, 2
    // or 3 of 8), so more than half as many; up to 256 take at most `alone` (7 of 4
    // elements).  No kernel is built for the others.
    if constexpr (kP <= (kN == 4 ? 7 : 4))
      if (sh.threads <= 256) return go(layer_norm_bwd_kernel<T, R, Y, kN, kP, kWhole, 256>);
    if constexpr (kP > (kN == 4 ? 2 : 1))
      if (sh.threads > 256) return go(layer_norm_bwd_kernel<T, R, Y, kN, kP, kWhole, 512>);
    return static_cast<int>(hipErrorInvalidValue);
  } else {
    hipLaunchKernelGGL((layer_norm_fwd_kernel<T, R, Y, kN, kP, kWhole>),
                       dim3(forward_groups(a.rows, sh)),
                       dim3(sh.threads), 0, s, a, sh.lanes);
    return static_cast<int>(hipGetLastError());
  }
}

template <typename T, typename R, typename Y, int kN, bool kWhole, bool kBack>
int launch_w(const LayerNormArgs &a, const Shape &sh, hipStream_t s) {
  switch (sh.per) {
    case 1: return launch_p<T, R, Y, kN, 1, kWhole, kBack>(a, sh, s);
    case 2: return launch_p<T, R, Y, kN, 2, kWhole, kBack>(a, sh, s);
    case 3: return launch_p<T, R, Y, kN, 3, kWhole, kBack>(a, sh, s);
    case 4: return launch_p<T, R, Y, kN, 4, kWhole, kBack>(a, sh, s);
  }
  if constexpr (kN == 4)
    if (sh.per == 5) return launch_p<T, R, Y, kN, 5, kWhole, kBack>(a, sh, s);
  if constexpr (kN == 4) {
    if (sh.per == 6) return launch_p<T, R, Y, kN, 6, kWhole, kBack>(a, sh, s);
    if (sh.per == 7) return launch_p<T, R, Y, kN, 7, kWhole, kBack>(a, sh, s);
    if (sh.per == 8) return launch_p<T, R, Y, kN, 8, kWhole, kBack>(a, sh, s);
  }
  return static_cast<int>(hipErrorInvalidValue);
}

template <typename T, typename R, typename Y, int kN, bool kBack>
int launch_n(const LayerNormArgs &a, const Shape &sh, hipStream_t s) {
  return sh.whole ? launch_w<T, R, Y, kN, true, kBack>(a, sh, s)
                  : launch_w<T, R, Y, kN, false, kBack>(a, sh, s);
}

template <bool kBack>
int launch(const LayerNormArgs &a, const Shape &sh, LayerNormTypes types, hipStream_t s) {
  switch (types) {
    case kLnBf16: return launch_n<uint16_t, uint16_t, uint16_t, 8, kBack>(a, sh, s);
    case kLnBf16Wide: return launch_n<uint16_t, float, uint16_t, 8, kBack>(a, sh, s);
    case kLnF32: return launch_n<float, float, float, 4, kBack>(a, sh, s);
    default: return launch_n<float, float, uint16_t, 8, kBack>(a, sh, s);
  }
}

}  // namespace

int layer_norm_bwd_parts(int64_t rows, int dim) {
  int most = 0;
  for (LayerNormTypes t : {kLnBf16, kLnBf16Wide, kLnF32, kLnF32Bf16}) {
    const int n = back_groups(rows, shape_of(dim, t, true), t);
    if (n > most) most = n;
  }
  return most;
}

int launch_layer_norm_fwd(const LayerNormArgs &a, LayerNormTypes types, void *stream) {
  return launch<false>(a, shape_of(a.dim, types, false), types, static_cast<hipStream_t>(stream));
}

int launch_layer_norm_bwd(const LayerNormArgs &args, LayerNormTypes types, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  LayerNormArgs a = args;
  a.nparts = 0;
  if (a.rows > 0) {
    const Shape sh = shape_of(a.dim, types, true);
    a.nparts = back_groups(a.rows, sh, types);
    const int err = launch<true>(a, sh, types, s);
    if (err != 0) return err;
  }
  if (!a.dweight && !a.dbias) return 0;
  hipLaunchKernelGGL(layer_norm_parts_kernel, dim3(static_cast<unsigned>((a.dim + 31) / 32), 2),
                     dim3(1024), 0, s, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
