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
constexpr int kAhead = 8;

__global__ __launch_bounds__(256) void linattn_chain_kernel(LinChain a, LinChain other) {
  const LinChain &p = blockIdx.z ? other : a;
  const int h = blockIdx.x % static_cast<unsigned>(p.plan.heads);
  const int seq = blockIdx.x / static_cast<unsigned>(p.plan.heads);
  int64_t b, e;
  sequence_rows(p.plan, seq, &b, &e);
  int64_t segs = (e - b + p.plan.seg_len - 1) / p.plan.seg_len;
  if (segs < 1) segs = 1;
  const int64_t i = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
  if (i >= p.size) return;
  const int64_t slot0 = first_slot(p.plan, seq) + (p.reverse ? segs - 1 : 0);
  const int64_t step = p.reverse ? -p.plan.heads : p.plan.heads;  // cells
  const int64_t cell0 = slot0 * p.plan.heads + h;
  float acc = p.first ? p.first[(static_cast<int64_t>(seq) * p.plan.heads + h) * p.size + i] : 0.0f;
  for (int64_t k = 0; k < segs; k += kAhead) {
    float add[kAhead], decay[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      // nothing reads what the last segment adds
      const bool in = k + j + 1 < segs;
      const int64_t cell = cell0 + (in ? k + j : 0) * step;
      add[j] = in ? p.states[cell * p.size + i] : 0.0f;
      decay[j] = in ? p.decay[cell] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k + j < segs) {
        p.states[(cell0 + (k + j) * step) * p.size + i] = acc;
        acc = fmaf(acc, decay[j], add[j]);
      }
  }
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

// Pairs inside each chunk: out_t = sum_{s<t} W_ts - sum_{r>t} W_rt.  One
// workgroup per (chunk, head); a wave takes 16 tokens t and half of the tokens
// s (bf16) or all (fp32).  Operands come from memory straight into fragments,
// 128 columns of all of them at once (latency bounds it: every row is read
// by few waves and used in 8 products).
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

template <typename T, bool kVec>
__global__ __launch_bounds__(512) void linattn_pairs_kernel(LinPairs p) {
  typedef Traits<T> Tr;
  typedef typename Tr::Frag Frag;
  constexpr int C = Tr::kChunk, kNT = C / 16;
  constexpr int kSub = Tr::kBf16 ? 2 : 1, kPer = kNT / kSub;  // tiles a wave, waves a tile row
  constexpr int kKS = 4;                                      // steps of 32 columns in flight
  __shared__ double As[C];
  __shared__ float Cols[kNT][C];
  __shared__ float Rows[kPer][C];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int h = blockIdx.x % static_cast<unsigned>(p.plan.heads);
  const unsigned per_seg = static_cast<unsigned>(p.plan.seg_len) / C;
  const unsigned cs = blockIdx.x / static_cast<unsigned>(p.plan.heads);
  const Segment sg = segment_of(p.plan, cs / per_seg);
  const int64_t t0 = sg.begin + static_cast<int64_t>(cs % per_seg) * C;
  if (!sg.real || t0 >= sg.end) return;
  const int rows = sg.end - t0 < C ? static_cast<int>(sg.end - t0) : C;
  const int ti = wave / kPer, s0 = wave % kPer * kSub;
  const bool some = s0 <= ti;  // else every pair of this wave's is empty
  f32x4 w[kSub];
#pragma unroll
  for (int si = 0; si < kSub; ++si) w[si] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (some) {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const LinSide &xr = part ? p.o : p.q, &xc = part ? p.v : p.k;
      const __amdgpu_buffer_rsrc_t vr = rows_view(
          static_cast<const T *>(xr.p) + t0 * xr.stride + (h / xr.div) * xr.d, xr.stride, rows, xr.d);
      const __amdgpu_buffer_rsrc_t vc = rows_view(
          static_cast<const T *>(xc.p) + t0 * xc.stride + (h / xc.div) * xc.d, xc.stride, rows, xc.d);
      f32x4 acc[kSub];
#pragma unroll
      for (int si = 0; si < kSub; ++si) acc[si] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int c0 = 0; c0 < xr.d; c0 += 32 * kKS) {
        Frag b[kKS], a[kKS][kSub];
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
          const int c = c0 + 32 * ks + 8 * lq;
          b[ks] = view_frag<T, kVec>(
              vr, static_cast<int>(((16 * ti + li) * xr.stride + c) * sizeof(T)), xr.d - c);
#pragma unroll
          for (int si = 0; si < kSub; ++si)
            a[ks][si] = view_frag<T, kVec>(
                vc, static_cast<int>(((16 * (s0 + si) + li) * xc.stride + c) * sizeof(T)),
                xc.d - c);
        }
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int si = 0; si < kSub; ++si) acc[si] = mma(a[ks][si], b[ks], acc[si]);
      }
#pragma unroll
      for (int si = 0; si < kSub; ++si) w[si] = part ? w[si] * acc[si] : acc[si];
    }
  }
  if (wave == 0) {
    const float g = lane < rows ? decay_at(p.g, p.g_kind, t0 + lane, p.plan.heads, h) : 0.0f;
    const double a = wave_sums<C>(lane < C ? log2_decay(g) : 0.0, lane);
    if (lane < C) As[lane] = a;
  }
  __syncthreads();
  // lane: token t = 16 ti + li against s = 16 (s0 + si) + 4 lq + e
  const int t = 16 * ti + li;
  const double at = As[t];
  float row_sum = 0.0f;
#pragma unroll
  for (int si = 0; si < kSub; ++si) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int s = 16 * (s0 + si) + 4 * lq + e;
      const float f = fast_exp2(static_cast<float>(at - As[s])) * p.scale;
      const float x = s < t ? w[si][e] * f : 0.0f;
      row_sum += x;
      float col = x;
      col += __shfl_xor(col, 1);
      col += __shfl_xor(col, 2);
      col += __shfl_xor(col, 4);
      col += __shfl_xor(col, 8);
      if (li == 0) Cols[ti][s] = col;
    }
  }
  row_sum += __shfl_xor(row_sum, 16);
  row_sum += __shfl_xor(row_sum, 32);
  if (lq == 0) Rows[wave % kPer][t] = row_sum;
  __syncthreads();
  if (tid < rows) {
    float c = 0.0f, r = 0.0f;
#pragma unroll
    for (int i = 0; i < kNT; ++i) c += Cols[i][tid];
#pragma unroll
    for (int i = 0; i < kPer; ++i) r += Rows[i][tid];
    p.out[(t0 + tid) * p.plan.heads + h] = r - c;
  }
}

// One workgroup per (segment, head): the inner product at the segment's end,
// then the sums from there backwards, in 64 bits.
__global__ __launch_bounds__(256) void linattn_decay_grad_kernel(LinDecayGrad p) {
  __shared__ double Red[4];
  __shared__ double Run[4][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x % p.plan.heads;
  const int64_t slot = blockIdx.x / p.plan.heads;
  const Segment sg = segment_of(p.plan, slot);
  if (!sg.real || sg.begin >= sg.end) return;
  const int64_t n = sg.end - sg.begin;
  // tokens from here on are summed from the state before them
  const int64_t tail = sg.last ? (n - 1) / p.chunk * p.chunk : n;
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
    for (int64_t i0 = tid; i0 < p.size; i0 += 256 * kFly) {
      float x[kFly], y[kFly];
#pragma unroll
      for (int j = 0; j < kFly; ++j) {
        const int64_t i = i0 + 256 * j;
        x[j] = i < p.size ? state[i] : 0.0f;
        y[j] = i < p.size ? adj[i] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kFly; ++j) dot += static_cast<double>(x[j]) * static_cast<double>(y[j]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d);
  if (lane == 0) Red[wave] = dot;
  __syncthreads();
  double end = (Red[0] + Red[1] + Red[2] + Red[3]) * factor;
  for (int64_t base = (n - 1) / 256 * 256; base >= 0; base -= 256) {
    // thread i takes token base + 255 - i: sums from the end are prefix sums
    const int64_t k = base + 255 - tid;
    double v = 0.0, y = 0.0;
    const int64_t at = (sg.begin + k) * p.plan.heads + h;
    if (k < n) {
      v = p.pairs[at];
      for (int s = 0; s < p.xslices; ++s) v += p.xdots[s * p.plan.tokens * p.plan.heads + at];
      for (int s = 0; s < p.yslices; ++s) y += p.ydots[s * p.plan.tokens * p.plan.heads + at];
      if (k < tail) {
        v -= y;
        y = 0.0;
      }
    }
    v = wave_sums<64>(v, lane);
    y = wave_sums<64>(y, lane);
    if (lane == 63) {
      Run[wave][0] = v;
      Run[wave][1] = y;
    }
    __syncthreads();
    double before = end, from = 0.0;  // sums over the tokens behind this wave's
    for (int w = 0; w < wave; ++w) {
      before += Run[w][0];
      from += Run[w][1];
    }
    const double all = end + Run[0][0] + Run[1][0] + Run[2][0] + Run[3][0];
    const double ally = Run[0][1] + Run[1][1] + Run[2][1] + Run[3][1];
    // columns of the tail's tokens before k (the others' are 0)
    const double columns = k >= tail ? ally - (from + y) : 0.0;
    if (k < n) p.dg[at] = static_cast<float>(before + v + columns);
    __syncthreads();
    end = all;
  }
}

// ------------------------------------------------------------ reductions ---
__device__ __forceinline__ void all_rows(const LinPlan &p, int64_t *begin, int64_t *end) {
  int64_t b, e, unused;
  sequence_rows(p, 0, begin, &unused);
  sequence_rows(p, p.nseq - 1, &b, &e);
  *end = e;
}

template <typename T>
__global__ __launch_bounds__(256) void linattn_head_sum_kernel(const float *in, T *out,
                                                               LinPlan plan, int div, int d) {
  int64_t begin, end;
  all_rows(plan, &begin, &end);
  const int64_t row = static_cast<int64_t>(plan.heads / div) * d;  // of out
  const int64_t stop = end * row, step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = begin * row + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < stop;
       i += step) {
    const int64_t t = i / row, c = i % row;
    const float *s = in + t * plan.heads * d + c / d * div * d + c % d;
    float acc = 0.0f;
    for (int k = 0; k < div; ++k) acc += s[static_cast<int64_t>(k) * d];
    out[i] = from_f32<T>(acc);
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

// ------------------------------------------------------------------ step ---
// One token: a workgroup takes 64 columns of one row's head state, 16
// threads with 4 neighbouring columns each in 16 groups over the state's
// rows.  The state is read and written once; everything else is small.
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
  const int64_t parts = (a.size + 255) / 256;
  hipLaunchKernelGGL(linattn_chain_kernel,
                     dim3(static_cast<unsigned>(a.plan.nseq * static_cast<int64_t>(a.plan.heads)),
                          static_cast<unsigned>(parts), b ? 2 : 1),
                     dim3(256), 0, static_cast<hipStream_t>(stream), a, b ? *b : a);
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_pairs(const LinPairs &a, bool bf16, void *stream) {
  const dim3 grid(
      static_cast<unsigned>(a.plan.slots * (a.plan.seg_len / a.chunk) * a.plan.heads));
  hipStream_t s = static_cast<hipStream_t>(stream);
  // 16 tiles in pairs, or 4: a wave each
  if (bf16) {
    if (a.plan.vec)
      hipLaunchKernelGGL((linattn_pairs_kernel<uint16_t, true>), grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((linattn_pairs_kernel<uint16_t, false>), grid, dim3(512), 0, s, a);
  } else {
    if (a.plan.vec)
      hipLaunchKernelGGL((linattn_pairs_kernel<float, true>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((linattn_pairs_kernel<float, false>), grid, dim3(256), 0, s, a);
  }
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_decay_grad(const LinDecayGrad &a, void *stream) {
  hipLaunchKernelGGL(linattn_decay_grad_kernel,
                     dim3(static_cast<unsigned>(a.plan.slots * a.plan.heads)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a);
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_head_sum(const float *in, void *out, const LinPlan &plan, int div, int d,
                            bool bf16, void *stream) {
  const int64_t n = plan.tokens * (plan.heads / div) * d, most = 1 << 16;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256 < most ? (n + 255) / 256 : most));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (bf16)
    hipLaunchKernelGGL(linattn_head_sum_kernel<uint16_t>, grid, dim3(256), 0, s, in,
                       static_cast<uint16_t *>(out), plan, div, d);
  else
    hipLaunchKernelGGL(linattn_head_sum_kernel<float>, grid, dim3(256), 0, s, in,
                       static_cast<float *>(out), plan, div, d);
  return static_cast<int>(hipGetLastError());
}

int launch_linattn_token_sum(const float *in, float *out, const LinPlan &plan, void *stream) {
  hipLaunchKernelGGL(linattn_token_sum_kernel, dim3(static_cast<unsigned>(plan.heads)), dim3(1024),
                     0, static_cast<hipStream_t>(stream), in, out, plan);
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
