// ssm_embed.hip -- gfx950 kernels of the embedding and of its gradient.
//
//   out_t = scale weight[ids_t]                    (0 for ids outside 0..vocab-1)
//   dweight_v (+)= scale sum_{t: ids_t = v} dy_t
//
// The gradient sorts the tokens by their id (a stable radix sort of (id,
// token) pairs, 8 bits a pass, so that tokens of one id stay in order) and
// cuts the sorted list into runs of equal length.  A wave sums one run's rows
// of dy, for the columns that its lanes hold, and writes the sum of every id
// that begins and ends in the run; the sums of ids that go on over a run's end
// go to a partial row each and are added by a second kernel.  No sum depends
// on an order that may change, and an id that half of all tokens have is
// spread over as many waves as there are runs of it.
#include "ssm_model_internal.h"
#include "ssm_pieces.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWavesPer = kThreads / 64;

// The id of a token as a sort key: vocab for ids outside.
__device__ __forceinline__ uint32_t key_of(const EmbedArgs &p, int64_t t) {
  const int64_t id = p.wide_ids ? static_cast<const int64_t *>(p.ids)[t]
                                : static_cast<const int32_t *>(p.ids)[t];
  return id >= 0 && id < p.vocab ? static_cast<uint32_t>(id) : static_cast<uint32_t>(p.vocab);
}

// ---------------------------------------------------------------- forward --
// A workgroup takes rows_per rows at a time, their pieces flat over its lanes.
template <typename W, typename T, int kN>
__global__ __launch_bounds__(kThreads) void embed_fwd_kernel(EmbedArgs p, int rows_per) {
  const uint32_t pieces = (p.dim + kN - 1) / kN;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_per; row0 < p.tokens;
       row0 += static_cast<int64_t>(gridDim.x) * rows_per) {
    const int64_t left = p.tokens - row0;
    const uint32_t all = pieces * static_cast<uint32_t>(left < rows_per ? left : rows_per);
    for (uint32_t l = threadIdx.x; l < all; l += kThreads) {
      const uint32_t r = l / pieces, q = l - r * pieces;
      const uint32_t key = key_of(p, row0 + r);
      float v[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) v[e] = 0.0f;
      if (key < p.vocab) {
        get_piece<W, kN>(static_cast<const W *>(p.weight) + key * p.w_stride, q, p.dim, v);
#pragma unroll
        for (int e = 0; e < kN; ++e) v[e] *= p.scale;
      }
      store_piece<T, kN>(static_cast<T *>(p.out) + (row0 + r) * p.dim, q, p.dim, v);
    }
  }
}

// ------------------------------------------------------------------- sort --
constexpr int kTile = 4096;             // tokens a workgroup sorts in a pass
constexpr int kPer = kTile / kThreads;  // keys a thread holds
constexpr int kBins = 256;

struct SortPass {
  const uint32_t *keys, *pos;  // null in the first pass: the ids themselves
  uint32_t *keys_out, *pos_out;
  uint32_t *counts;            // (bins, tiles)
  int64_t tiles;
  int shift;
};

// Keys of the pass that the thread holds: a wave's are neighbours, 64 at a time.
__device__ __forceinline__ int64_t sort_index(int64_t tile, int i) {
  return tile * kTile + (threadIdx.x >> 6) * (64 * kPer) + i * 64 + (threadIdx.x & 63);
}
__device__ __forceinline__ uint32_t sort_key(const EmbedArgs &p, const SortPass &s, int64_t at) {
  return s.keys ? s.keys[at] : key_of(p, at);
}

__global__ __launch_bounds__(kThreads) void embed_count_kernel(EmbedArgs p, SortPass s) {
  __shared__ uint32_t Count[kBins];
  for (int64_t tile = blockIdx.x; tile < s.tiles; tile += gridDim.x) {
    Count[threadIdx.x] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t at = sort_index(tile, i);
      if (at < p.tokens) atomicAdd(&Count[sort_key(p, s, at) >> s.shift & 255u], 1u);
    }
    __syncthreads();
    s.counts[threadIdx.x * s.tiles + tile] = Count[threadIdx.x];
    __syncthreads();
  }
}

// Counts before each (bin, tile), in that order: one workgroup.
__global__ __launch_bounds__(1024) void embed_offsets_kernel(SortPass s) {
  __shared__ uint32_t Sums[16];
  const int64_t n = kBins * s.tiles;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t before = 0u;
  for (int64_t base = 0; base < n; base += 4096) {
    uint32_t c[4], sum = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = base + 4 * threadIdx.x + i;
      c[i] = at < n ? s.counts[at] : 0u;
      sum += c[i];
    }
    uint32_t up = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t o = __shfl_up(up, d);
      if (lane >= d) up += o;
    }
    if (lane == 63) Sums[wave] = up;
    __syncthreads();
    uint32_t mine = before + up - sum, all = 0u;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) mine += Sums[w];
      all += Sums[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = base + 4 * threadIdx.x + i;
      if (at < n) s.counts[at] = mine;
      mine += c[i];
    }
    before += all;
    __syncthreads();
  }
}

// Lanes of the wave whose 8-bit digit is this lane's, among those in `in`.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, uint64_t in) {
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool bit = digit >> b & 1u;
    const uint64_t set = __ballot(bit);
    in &= bit ? set : ~set;
  }
  return in;
}

__global__ __launch_bounds__(kThreads) void embed_scatter_kernel(EmbedArgs p, SortPass s) {
  __shared__ uint32_t Count[kWavesPer][kBins];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t tile = blockIdx.x; tile < s.tiles; tile += gridDim.x) {
#pragma unroll
    for (int w = 0; w < kWavesPer; ++w) Count[w][threadIdx.x] = 0u;
    __syncthreads();
    uint32_t key[kPer], rank[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t at = sort_index(tile, i);
      const bool in = at < p.tokens;
      key[i] = in ? sort_key(p, s, at) : 0u;
      const uint32_t digit = key[i] >> s.shift & 255u;
      const uint64_t same = same_digit(digit, __ballot(in));
      const int first = __ffsll(static_cast<unsigned long long>(same)) - 1;
      uint32_t old = 0u;
      if (in && lane == first)
        old = atomicAdd(&Count[wave][digit], static_cast<uint32_t>(__popcll(same)));
      old = __shfl(old, first < 0 ? 0 : first);
      rank[i] = old + __popcll(same & ((uint64_t(1) << lane) - 1));
    }
    __syncthreads();
    {
      // places of the tile's keys with this thread's digit, wave after wave
      uint32_t at = s.counts[threadIdx.x * s.tiles + tile];
#pragma unroll
      for (int w = 0; w < kWavesPer; ++w) {
        const uint32_t c = Count[w][threadIdx.x];
        Count[w][threadIdx.x] = at;
        at += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t at = sort_index(tile, i);
      if (at < p.tokens) {
        const uint32_t to = Count[wave][key[i] >> s.shift & 255u] + rank[i];
        s.keys_out[to] = key[i];
        s.pos_out[to] = s.pos ? s.pos[at] : static_cast<uint32_t>(at);
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- sums --
struct Runs {
  const uint32_t *keys, *pos;  // sorted
  float *parts;                // (runs, 2, columns)
  int64_t runs, row;           // elements of a partial row
  int len;                     // sorted tokens a run has, at most 64
};

// Whether the ids of sorted tokens i and i + 1 differ or the list ends there.
__device__ __forceinline__ bool ends_at(const EmbedArgs &p, const Runs &r, int64_t i) {
  return i + 1 >= p.tokens || r.keys[i + 1] != r.keys[i];
}

template <typename W, int kN>
__device__ __forceinline__ void put_sum(const EmbedArgs &p, uint32_t key, int q, float (&v)[kN]) {
  W *row = static_cast<W *>(p.dweight) + static_cast<int64_t>(key) * p.dim;
#pragma unroll
  for (int e = 0; e < kN; ++e) v[e] *= p.scale;
  if (p.accumulate) {
    float old[kN];
    get_piece<W, kN>(row, q, p.dim, old);
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] += old[e];
  }
  store_piece<W, kN>(row, q, p.dim, v);
}

// A wave takes one run and 64 pieces of the columns.
template <typename T, typename W, int kN>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(EmbedArgs p, Runs r) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t run = static_cast<int64_t>(blockIdx.x) * kWavesPer + wave;
  if (run >= r.runs) return;
  const int pieces = (p.dim + kN - 1) / kN;
  const int q = blockIdx.y * 64 + lane;
  const int64_t from = run * r.len;
  const int n = static_cast<int>(p.tokens - from < r.len ? p.tokens - from : r.len);
  uint32_t key = 0u, pos = 0u;
  bool end = false;
  if (lane < n) {
    key = r.keys[from + lane];
    pos = r.pos[from + lane];
    end = ends_at(p, r, from + lane);
  }
  const uint64_t ends = __ballot(end);
  // the first id may have begun in a run before
  bool came = from > 0 && r.keys[from - 1] == __shfl(key, 0);
  float acc[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) acc[e] = 0.0f;
  float *part = r.parts + run * 2 * r.row;
  for (int j = 0; j < n; j += kAhead) {
    Piece<T, kN> dy[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int at = j + k < n ? j + k : n - 1;
      const int64_t t = static_cast<uint32_t>(__builtin_amdgcn_readlane(pos, at));
      dy[k].zero();
      if (q < pieces) load_piece(dy[k], static_cast<const T *>(p.dy) + t * p.dy_stride, q, p.dim);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (j + k >= n) break;
      const uint32_t id = __builtin_amdgcn_readlane(key, j + k);
#pragma unroll
      for (int e = 0; e < kN; ++e) acc[e] += dy[k][e];
      const bool stop = ends >> (j + k) & 1;
      if (!stop && j + k < n - 1) continue;
      if (id < p.vocab && q < pieces) {
        if (stop && !came)
          put_sum<W, kN>(p, id, q, acc);
        else
          store_piece<float, kN>(part + (came ? 0 : r.row), q, p.dim, acc);
      }
      came = false;
#pragma unroll
      for (int e = 0; e < kN; ++e) acc[e] = 0.0f;
    }
  }
}

// The run in which an id begins that goes on behind it adds the partial rows
// of that id.  A workgroup a run and 64 pieces of the columns; its waves take
// the partial rows in turn.
template <typename W, int kN>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedArgs p, Runs r) {
  __shared__ float Sums[kWavesPer][kN][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t run = blockIdx.x;
  const int64_t last = (run + 1) * r.len - 1;
  if (last >= p.tokens - 1) return;
  const uint32_t key = r.keys[last];
  if (key >= p.vocab || r.keys[last + 1] != key) return;
  const int64_t from = run * r.len;
  if (r.keys[from] == key && from > 0 && r.keys[from - 1] == key) return;
  const int pieces = (p.dim + kN - 1) / kN;
  const int q = blockIdx.y * 64 + lane;
  float acc[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) acc[e] = 0.0f;
  if (q < pieces) {
    if (wave == 0) get_piece<float, kN>(r.parts + (run * 2 + 1) * r.row, q, p.dim, acc);
    for (int64_t c = run + 1 + wave; c < r.runs && r.keys[c * r.len] == key; c += kWavesPer) {
      float v[kN];
      get_piece<float, kN>(r.parts + c * 2 * r.row, q, p.dim, v);
#pragma unroll
      for (int e = 0; e < kN; ++e) acc[e] += v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < kN; ++e) Sums[wave][e][lane] = acc[e];
  __syncthreads();
  if (wave == 0 && q < pieces) {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      acc[e] = (Sums[0][e][lane] + Sums[1][e][lane]) + (Sums[2][e][lane] + Sums[3][e][lane]);
    put_sum<W, kN>(p, key, q, acc);
  }
}

// Zeros in the rows of ids that do not come.  A wave takes 32 rows; lane l
// finds where id l of them begins in the sorted list.
template <typename W>
__global__ __launch_bounds__(kThreads) void embed_clear_kernel(EmbedArgs p, const uint32_t *keys) {
  const int lane = threadIdx.x & 63;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kWavesPer + (threadIdx.x >> 6)) * 32;
  const int64_t want = row0 + (lane < 32 ? lane : 32);
  int64_t lo = 0, hi = p.tokens;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (keys[mid] < want)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int64_t next = __shfl_down(lo, 1);
  const uint64_t there = __ballot(lane < 32 && next > lo);
  constexpr int kN = 16 / sizeof(W);
  const int pieces = (p.dim + kN - 1) / kN;
  float zero[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) zero[e] = 0.0f;
  for (int k = 0; k < 32 && row0 + k < p.vocab; ++k) {
    if (there >> k & 1) continue;
    W *row = static_cast<W *>(p.dweight) + (row0 + k) * p.dim;
    for (int q = lane; q < pieces; q += 64) store_piece<W, kN>(row, q, p.dim, zero);
  }
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Sorted tokens a run has.
constexpr int kRunLen = 32;

// Workspace: two lists of keys and positions, the counts, the partial rows.
struct Layout {
  int64_t tiles, runs, row;
  int len;
  int64_t keys[2], pos[2], counts, parts, bytes;
};
Layout layout_of(int64_t tokens, int64_t dim) {
  Layout l;
  l.tiles = (tokens + kTile - 1) / kTile;
  l.len = kRunLen;
  l.runs = (tokens + l.len - 1) / l.len;
  l.row = up(dim, 4);
  int64_t at = 0;
  for (int i = 0; i < 2; ++i) {
    l.keys[i] = at;
    at += up(tokens * 4, 256);
    l.pos[i] = at;
    at += up(tokens * 4, 256);
  }
  l.counts = at;
  at += up(l.tiles * kBins * 4, 256);
  l.parts = at;
  at += l.runs > 1 ? l.runs * 2 * l.row * 4 : 0;
  l.bytes = at;
  return l;
}

template <typename T, typename W, int kN>
int launch_bwd(const EmbedArgs &a, hipStream_t s) {
  if (a.tokens == 0) {
    if (a.accumulate) return 0;
    hipLaunchKernelGGL(embed_clear_kernel<W>, dim3((a.vocab + 127) / 128), dim3(kThreads), 0, s, a,
                       nullptr);
    return static_cast<int>(hipGetLastError());
  }
  const Layout l = layout_of(a.tokens, a.dim);
  char *ws = static_cast<char *>(a.workspace);
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t *>(ws + at); };
  SortPass sort{nullptr, nullptr, words(l.keys[0]), words(l.pos[0]), words(l.counts), l.tiles, 0};
  const dim3 grid(static_cast<unsigned>(l.tiles < 65536 ? l.tiles : 65536));
  int to = 0;
  for (int shift = 0; shift == 0 || a.vocab >> shift != 0; shift += 8) {
    sort.shift = shift;
    sort.keys_out = words(l.keys[to]);
    sort.pos_out = words(l.pos[to]);
    hipLaunchKernelGGL(embed_count_kernel, grid, dim3(kThreads), 0, s, a, sort);
    hipLaunchKernelGGL(embed_offsets_kernel, dim3(1), dim3(1024), 0, s, sort);
    hipLaunchKernelGGL(embed_scatter_kernel, grid, dim3(kThreads), 0, s, a, sort);
    sort.keys = sort.keys_out;
    sort.pos = sort.pos_out;
    to ^= 1;
  }
  const Runs r{sort.keys, sort.pos, reinterpret_cast<float *>(ws + l.parts), l.runs, l.row, l.len};
  const unsigned cols = static_cast<unsigned>(((a.dim + kN - 1) / kN + 63) / 64);
  hipLaunchKernelGGL((embed_sum_kernel<T, W, kN>),
                     dim3(static_cast<unsigned>((l.runs + kWavesPer - 1) / kWavesPer), cols),
                     dim3(kThreads), 0, s, a, r);
  if (l.runs > 1)
    hipLaunchKernelGGL((embed_join_kernel<W, kN>), dim3(static_cast<unsigned>(l.runs), cols),
                       dim3(kThreads), 0, s, a, r);
  if (!a.accumulate)
    hipLaunchKernelGGL(embed_clear_kernel<W>, dim3(static_cast<unsigned>((a.vocab + 127) / 128)),
                       dim3(kThreads), 0, s, a, r.keys);
  return static_cast<int>(hipGetLastError());
}

template <typename W, typename T, int kN>
int launch_fwd(const EmbedArgs &a, hipStream_t s) {
  const int pieces = (a.dim + kN - 1) / kN;
  const int rows_per = pieces >= 512 ? 1 : 512 / pieces;
  const int64_t groups = (a.tokens + rows_per - 1) / rows_per;
  hipLaunchKernelGGL((embed_fwd_kernel<W, T, kN>),
                     dim3(static_cast<unsigned>(groups < (1 << 20) ? groups : 1 << 20)),
                     dim3(kThreads), 0, s, a, rows_per);
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int64_t embed_bwd_workspace(int64_t tokens, int64_t, int64_t dim) {
  return layout_of(tokens, dim).bytes;
}

int launch_embed_fwd(const EmbedArgs &a, bool w_bf16, bool bf16, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (w_bf16)
    return bf16 ? launch_fwd<uint16_t, uint16_t, 8>(a, s) : launch_fwd<uint16_t, float, 8>(a, s);
  return bf16 ? launch_fwd<float, uint16_t, 8>(a, s) : launch_fwd<float, float, 4>(a, s);
}

int launch_embed_bwd(const EmbedArgs &a, bool w_bf16, bool bf16, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (bf16)
    return w_bf16 ? launch_bwd<uint16_t, uint16_t, 8>(a, s) : launch_bwd<uint16_t, float, 8>(a, s);
  return w_bf16 ? launch_bwd<float, uint16_t, 8>(a, s) : launch_bwd<float, float, 4>(a, s);
}

}  // namespace ssm
