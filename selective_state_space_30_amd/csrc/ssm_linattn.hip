// ssm_linattn.hip -- linear attention with a decay for each head: the small
// kernels around the chunk kernel (ssm_linattn_core.h) and the single-token
// step.
#include "ssm_linattn_core.h"

namespace ssm {
namespace {

using namespace lin;

// ------------------------------------------------------- segment states ---
// Per (sequence, head): what each segment adds to the state -> the state
// that enters it, one segment after another.  A thread carries one element;
// kAhead segments are requested at once, so that the latency of memory is
// paid once for all of them.
// The first segment's state is the sequence's own, which its readers take
// from there.  kElems elements a thread: 1, or 4 where there are workgroups
// enough: 24 packed prompts of 16 heads, 68 us with 1 and 15 us with 4 (most
// are sequences of one or two segments); 8 heads of one sequence of 64
// segments, 25 us with 1 (its latency, 8 segments a trip).
constexpr int kAhead = 8;

template <int kElems>
__global__ __launch_bounds__(256) void linattn_chain_kernel(LinChain a, LinChain other) {
  const LinChain &p = blockIdx.z ? other : a;
  const int h = blockIdx.x % static_cast<unsigned>(p.plan.heads);
  const int seq = blockIdx.x / static_cast<unsigned>(p.plan.heads);
  int64_t b, e;
  sequence_rows(p.plan, seq, &b, &e);
  const int segs = static_cast<int>((static_cast<unsigned>(e - b) +
                                     static_cast<unsigned>(p.plan.seg_len) - 1) /
                                    static_cast<unsigned>(p.plan.seg_len));
  if (segs < 2) return;
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * 256 * kElems + threadIdx.x;
  const int64_t slot0 = first_slot(p.plan, seq) + (p.reverse ? segs - 1 : 0);
  const int64_t step = p.reverse ? -p.plan.heads : p.plan.heads;  // cells
  const int64_t cell0 = slot0 * p.plan.heads + h;
  const float *first =
      p.first ? p.first + (static_cast<int64_t>(seq) * p.plan.heads + h) * p.size : nullptr;
  float acc[kElems];
#pragma unroll
  for (int j = 0; j < kElems; ++j)
    acc[j] = first && i0 + 256 * j < p.size ? first[i0 + 256 * j] : 0.0f;
  for (int k = 0; k < segs; k += kAhead) {
    float add[kAhead][kElems], decay[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool in = k + u + 1 < segs;  // nothing reads what the last segment adds
      const int64_t cell = cell0 + (in ? k + u : 0) * step;
      decay[u] = in ? p.decay[cell] : 0.0f;
#pragma unroll
      for (int j = 0; j < kElems; ++j)
        add[u][j] = in && i0 + 256 * j < p.size ? p.states[cell * p.size + i0 + 256 * j] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k + u < segs) {
        float *s = p.states + (cell0 + (k + u) * step) * p.size;
#pragma unroll
        for (int j = 0; j < kElems; ++j) {
          if (k + u > 0 && i0 + 256 * j < p.size) s[i0 + 256 * j] = acc[j];
          acc[j] = fmaf(acc[j], decay[u], add[u][j]);
        }
      }
  }
}

// -------------------------------------------------- gradient of the decay ---
// One workgroup per (segment, head): the inner product at the segment's end,
// then the sums from there backwards, in 64 bits, a thread a token (a segment
// has at most 1024).  Measured: 16 heads, 4096 tokens in 10 segments, states of
// 128 x 128, 11 us (21 MB of states: latency of one trip).
constexpr int kGradThreads = 1024;

__global__ __launch_bounds__(kGradThreads) void linattn_decay_grad_kernel(LinDecayGrad p) {
  constexpr int kWaves = kGradThreads / 64;
  __shared__ double Red[kWaves];
  __shared__ double Run[kWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x % static_cast<unsigned>(p.plan.heads);
  const int64_t slot = blockIdx.x / static_cast<unsigned>(p.plan.heads);
  const Segment sg = segment_of(p.plan, slot);
  if (!sg.real || sg.begin >= sg.end) return;
  const int n = static_cast<int>(sg.end - sg.begin);
  // tokens from here on are summed from the state before them
  const int tail = sg.last ? (n - 1) / p.chunk * p.chunk : n;
  // thread i takes token n - 1 - i: sums from the end are prefix sums
  const int k = n - 1 - tid;
  const int64_t at = (sg.begin + k) * p.plan.heads + h;
  float pair = 0.0f, xs[2] = {0.0f, 0.0f}, ys[2] = {0.0f, 0.0f};
  if (k >= 0) {
    const int64_t all = p.plan.tokens * p.plan.heads;
    pair = p.pairs[at];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s < p.slices) {
        xs[s] = p.xdots[s * all + at];
        ys[s] = p.ydots[s * all + at];
      }
  }
  const float *state = nullptr, *adj = nullptr;
  const int64_t by_seq = (static_cast<int64_t>(sg.seq) * p.plan.heads + h) * p.size;
  double factor = 1.0;
  if (sg.last) {
    if (p.dlast) {
      state = p.last + by_seq;
      adj = p.dlast + by_seq;
      const int64_t t = sg.begin + tail + lane;  // (a chunk has at most 64 tokens)
      double sum = t < sg.end ? log2_decay(decay_at(p.g, p.g_kind, t, p.plan.heads, h)) : 0.0;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
      factor = fast_exp2(static_cast<float>(sum));
    }
  } else {
    state = p.states + ((slot + 1) * p.plan.heads + h) * p.size;
    adj = p.adjoints + (slot * p.plan.heads + h) * p.size;
  }
  double dot = 0.0;
  if (state) {
    // 16 elements of both in flight a thread (latency, not bytes)
    constexpr int kFly = 16;
    for (int i0 = tid; i0 < p.size; i0 += kGradThreads * kFly) {
      float x[kFly], y[kFly];
#pragma unroll
      for (int j = 0; j < kFly; ++j) {
        const int i = i0 + kGradThreads * j;
        x[j] = i < p.size ? state[i] : 0.0f;
        y[j] = i < p.size ? adj[i] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kFly; ++j) dot += static_cast<double>(x[j]) * static_cast<double>(y[j]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d);
  double v = static_cast<double>(pair) + xs[0] + xs[1];
  double y = static_cast<double>(ys[0]) + ys[1];
  if (k < tail) {
    v -= y;
    y = 0.0;
  }
  v = wave_sums<64>(v, lane);
  y = wave_sums<64>(y, lane);
  if (lane == 63) {
    Red[wave] = dot;
    Run[wave][0] = v;
    Run[wave][1] = y;
  }
  __syncthreads();
  double end = 0.0, before = 0.0, from = 0.0, ally = 0.0;
  for (int w = 0; w < kWaves; ++w) {
    end += Red[w];
    ally += Run[w][1];
    if (w < wave) {  // sums over the tokens behind this wave's
      before += Run[w][0];
      from += Run[w][1];
    }
  }
  // columns of the tail's tokens before k (the others' are 0)
  const double columns = k >= tail ? ally - (from + y) : 0.0;
  if (k >= 0) p.dg[at] = static_cast<float>(end * factor + before + v + columns);
}

// ------------------------------------------------------------ reductions ---
__device__ __forceinline__ void all_rows(const LinPlan &p, int64_t *begin, int64_t *end) {
  int64_t b, e, unused;
  sequence_rows(p, 0, begin, &unused);
  sequence_rows(p, p.nseq - 1, &b, &e);
  *end = e;
}

// Sums of `div` consecutive heads' fp32 rows, of dq's and dk's partial
// results at once (blockIdx.y); 4 neighbouring elements a thread where the
// head size allows, 8 heads' loads in flight (8000 tokens, 24 heads to one of 128: 29
// us, 6.8 TB/s, some of it from the last cache; 61 us with single elements and
// one load after the other).
template <typename T, int kN>
__global__ __launch_bounds__(256) void linattn_head_sum_kernel(const float *in0, const float *in1,
                                                               T *out0, T *out1, LinPlan plan,
                                                               int div, int d) {
  const float *in = blockIdx.y ? in1 : in0;
  T *out = blockIdx.y ? out1 : out0;
  int64_t begin, end;
  all_rows(plan, &begin, &end);
  const unsigned row = static_cast<unsigned>(plan.heads / div) * d / kN;  // pieces of an out row
  const unsigned per_head = static_cast<unsigned>(d) / kN;
  for (int64_t t = begin + blockIdx.x; t < end; t += gridDim.x)
    for (unsigned c = threadIdx.x; c < row; c += 256) {
      const float *s = in + t * plan.heads * d +
                       static_cast<int64_t>(c / per_head) * div * d + c % per_head * kN;
      float acc[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) acc[e] = 0.0f;
#pragma unroll 8
      for (int k = 0; k < div; ++k) {
        if constexpr (kN == 4) {
          const f32x4 x = *reinterpret_cast<const f32x4 *>(s + k * d);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += x[e];
        } else {
          acc[0] += s[k * d];
        }
      }
      T *o = out + (t * row + c) * kN;
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] = from_f32<T>(acc[e]);
    }
}

__global__ __launch_bounds__(1024) void linattn_token_sum_kernel(const float *in, float *out,
                                                                 LinPlan plan) {
  __shared__ double Red[1024];
  const int tid = threadIdx.x, h = blockIdx.x;
  int64_t begin, end;
  all_rows(plan, &begin, &end);
  double acc = 0.0;
  for (int64_t t = begin + tid; t < end; t += 1024) acc += in[t * plan.heads + h];
  Red[tid] = acc;
  __syncthreads();
  for (int d = 512; d > 0; d >>= 1) {
    if (tid < d) Red[tid] += Red[tid + d];
    __syncthreads();
  }
  if (tid == 0) out[h] = static_cast<float>(Red[0]);
}

// ------------------------------------------------- rows of no sequence ---
// Rows before the first and behind the last sequence of one array
// (blockIdx.y).  Rows start on any element: 16 bytes at a time between the
// first and the last such boundary, and 2 before and behind.
__global__ __launch_bounds__(256) void linattn_zero_outside_kernel(LinZero z) {
  char *base = static_cast<char *>(z.arrays[blockIdx.y].p);
  const int64_t row = z.arrays[blockIdx.y].row_bytes;
  int64_t begin, end;
  all_rows(z.plan, &begin, &end);
  const int64_t first = blockIdx.x * 256 + threadIdx.x, step = gridDim.x * 256;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base) + (side ? end : 0) * row;
    const uintptr_t hi = reinterpret_cast<uintptr_t>(base) + (side ? z.plan.tokens : begin) * row;
    uintptr_t a = (lo + 15) / 16 * 16, b = hi / 16 * 16;
    if (a > b) a = b = hi;  // inside one piece of 16 bytes
    for (uintptr_t p = lo + 2 * first; p < a; p += 2 * step) *reinterpret_cast<uint16_t *>(p) = 0;
    for (uintptr_t p = a + 16 * first; p < b; p += 16 * step)
      *reinterpret_cast<u32x4 *>(p) = u32x4{0u, 0u, 0u, 0u};
    for (uintptr_t p = b + 2 * first; p < hi; p += 2 * step) *reinterpret_cast<uint16_t *>(p) = 0;
  }
}

// ------------------------------------------------------------------ step ---
// One token: a workgroup takes 64 columns of one row's head state, 16
// threads with 4 neighbouring columns each in 16 groups over the state's
// rows.  The state is read and written once; everything else is small, so all
// of a thread's state is asked for before any of it is used.  Measured: 256
// rows of 16 heads of 128 x 128 (some idle), 505 MB: 88 us on states that the
// caches hold in part, 112 us a call on others (4.5 TB/s; a large copy: 5.2);
// one row of 80 heads of 128 x 64, 6 us (latency).
constexpr int kStepCols = 64, kStepGroups = 16;
constexpr int kStepRows = kLinMaxDim / kStepGroups;  // state rows a thread may take

template <typename T, bool kVec>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinStep p) {
  __shared__ float Qs[kLinMaxDim], Ks[kLinMaxDim];
  __shared__ __align__(16) float Part[kStepGroups][kStepCols];
  const int tid = threadIdx.x;
  const int slices = (p.dv + kStepCols - 1) / kStepCols;
  const int slice = blockIdx.x % slices;
  const int h = blockIdx.x / slices % p.heads;
  const int64_t b = blockIdx.x / slices / p.heads;
  const int hk = h / (p.heads / p.qk_heads);
  const int64_t slot = p.slot_of ? p.slot_of[b] : b;
  // a row without a slot of its own: out of range, or an earlier row's
  int taken = slot < 0 || slot >= p.slots;
  if (p.slot_of && !taken)
    for (int64_t i = tid; i < b; i += 256) taken |= p.slot_of[i] == slot;
  if (tid < p.dk) {
    const int64_t at = static_cast<int64_t>(hk) * p.dk + tid;
    Qs[tid] = to_f32<T>(static_cast<const T *>(p.q)[b * p.q_stride + at]);
    Ks[tid] = to_f32<T>(static_cast<const T *>(p.k)[b * p.k_stride + at]);
  }
  taken = __syncthreads_or(taken);
  const int cg = tid & 15, rg = tid >> 4;
  const int c = slice * kStepCols + 4 * cg;   // this thread's first column
  T *o = static_cast<T *>(p.o) + (b * p.heads + h) * p.dv;
  if (taken) {
    if (tid < kStepCols && slice * kStepCols + tid < p.dv)
      o[slice * kStepCols + tid] = from_f32<T>(0.0f);
    return;
  }
  const float decay =
      p.g_kind == kLinDecayNone
          ? 1.0f
          : fast_exp2(static_cast<float>(log2_decay(
                p.g_kind == kLinDecayHead ? p.g[h] : p.g[b * p.heads + h])));
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = c + e < p.dv
               ? to_f32<T>(static_cast<const T *>(
                     p.v)[b * p.v_stride + static_cast<int64_t>(h) * p.dv + c + e])
               : 0.0f;
  float *s = p.state + (slot * p.heads + h) * p.dk * p.dv + c;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  f32x4 x[kStepRows];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int r = rg + kStepGroups * i;
    x[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (r < p.dk && c < p.dv) {
      if (kVec) {
        x[i] = *reinterpret_cast<const f32x4 *>(s + r * p.dv);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.dv) x[i][e] = s[r * p.dv + e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int r = rg + kStepGroups * i;
    if (r < p.dk && c < p.dv) {
      const float k = Ks[r], q = Qs[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[i][e] = fmaf(x[i][e], decay, k * v[e]);
        acc[e] = fmaf(q, x[i][e], acc[e]);
      }
      if (kVec) {
        *reinterpret_cast<f32x4 *>(s + r * p.dv) = x[i];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.dv) s[r * p.dv + e] = x[i][e];
      }
    }
  }
  *reinterpret_cast<f32x4 *>(&Part[rg][4 * cg]) = acc;
  __syncthreads();
  if (tid < kStepCols && slice * kStepCols + tid < p.dv) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kStepGroups; ++i) sum += Part[i][tid];
    o[slice * kStepCols + tid] = from_f32<T>(sum * p.scale);
  }
}

}  // namespace

int linattn_chunk(bool bf16) { return bf16 ? kLinChunkBf16 : kLinChunkF32; }

int linattn_slice(int dv) { return dv > 64 ? 128 : 64; }

bool linattn_pairs_heads(int div, int dv) { return dv <= 64 && div % 2 == 0; }

int launch_linattn_chain(const LinChain &a, const LinChain *b, void *stream) {
  const int64_t cells = a.plan.nseq * static_cast<int64_t>(a.plan.heads);
  const int64_t parts = (a.size + 255) / 256;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (cells * parts > 4096)
    hipLaunchKernelGGL(linattn_chain_kernel<4>,
                       dim3(static_cast<unsigned>(cells), static_cast<unsigned>((parts + 3) / 4),
                            b ? 2 : 1),
                       dim3(256), 0, s, a, b ? *b : a);
  else
    hipLaunchKernelGGL(linattn_chain_kernel<1>,
                       dim3(static_cast<unsigned>(cells), static_cast<unsigned>(parts), b ? 2 : 1),
                       dim3(256), 0, s, a, b ? *b : a);
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_decay_grad(const LinDecayGrad &a, void *stream) {
  hipLaunchKernelGGL(linattn_decay_grad_kernel,
                     dim3(static_cast<unsigned>(a.plan.slots * a.plan.heads)), dim3(kGradThreads),
                     0, static_cast<hipStream_t>(stream), a);
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_head_sum(const float *in0, const float *in1, void *out0, void *out1,
                            const LinPlan &plan, int div, int d, bool bf16, void *stream) {
  const int64_t most = 1 << 16;
  const dim3 grid(static_cast<unsigned>(plan.tokens < most ? plan.tokens : most), 2);
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto kernel, auto *o0, auto *o1) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, in0, in1, o0, o1, plan, div, d);
    return static_cast<int>(hipGetLastError());
  };
  if (bf16) {
    uint16_t *o0 = static_cast<uint16_t *>(out0), *o1 = static_cast<uint16_t *>(out1);
    return d % 4 == 0 ? go(linattn_head_sum_kernel<uint16_t, 4>, o0, o1)
                      : go(linattn_head_sum_kernel<uint16_t, 1>, o0, o1);
  }
  float *o0 = static_cast<float *>(out0), *o1 = static_cast<float *>(out1);
  return d % 4 == 0 ? go(linattn_head_sum_kernel<float, 4>, o0, o1)
                    : go(linattn_head_sum_kernel<float, 1>, o0, o1);
}

int launch_linattn_token_sum(const float *in, float *out, const LinPlan &plan, void *stream) {
  hipLaunchKernelGGL(linattn_token_sum_kernel, dim3(static_cast<unsigned>(plan.heads)), dim3(1024),
                     0, static_cast<hipStream_t>(stream), in, out, plan);
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_zero_outside(const LinZero &a, void *stream) {
  unsigned arrays = 0;
  for (const auto &x : a.arrays) arrays += x.p != nullptr;
  hipLaunchKernelGGL(linattn_zero_outside_kernel, dim3(256, arrays), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a);
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_step(const LinStep &a, bool bf16, void *stream) {
  const int64_t slices = (a.dv + kStepCols - 1) / kStepCols;
  const dim3 grid(static_cast<unsigned>(a.batch * a.heads * slices));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool vec = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
  if (bf16) {
    if (vec)
      hipLaunchKernelGGL((linattn_step_kernel<uint16_t, true>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((linattn_step_kernel<uint16_t, false>), grid, dim3(256), 0, s, a);
  } else {
    if (vec)
      hipLaunchKernelGGL((linattn_step_kernel<float, true>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((linattn_step_kernel<float, false>), grid, dim3(256), 0, s, a);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
