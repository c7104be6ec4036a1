// ssm_embed.hip -- gfx950 kernels of the embedding and of its gradient.
//
//   out_t = scale weight[ids_t]                    (0 for ids outside 0..vocab-1)
//   dweight_v (+)= scale sum_{t: ids_t = v} dy_t
//
// The gradient sorts the tokens by their id (a stable radix sort of (id,
// token) pairs, digits of up to 9 bits, so that tokens of one id stay in order) and
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

// The id of a token as a sort key: vocab for ids outside.  Both words of a wide
// id are read as words, the only one of a narrow id twice: without a branch, at
// whose end the compiler would wait for each load.
__device__ __forceinline__ uint32_t key_of(const EmbedArgs &p, int64_t t) {
  const uint32_t *word = static_cast<const uint32_t *>(p.ids) + (t << p.wide_ids);
  const uint32_t low = word[0], high = word[p.wide_ids] & (0u - p.wide_ids);
  return high == 0u && low < static_cast<uint32_t>(p.vocab) ? low : static_cast<uint32_t>(p.vocab);
}

// ---------------------------------------------------------------- forward --
// A group of `lanes` (8..64) neighbouring lanes takes a row, kAhead pieces a
// lane in flight, and then the row `step` rows behind, whose id it has asked
// for before.  Bound by memory: 16384 tokens of 2560 columns of 50000, bf16
// into fp32, 50 us.  168 MB are written, which alone take 32 us (as rows of
// zeros), and 57 MB come from memory for the 32 MB of rows that occur: what is
// written pushes them out of the caches.  Stores that pass the caches by make it
// 33 us in a loop of such calls, but the norm behind it then reads the rows from
// memory: behind other work 120 us instead of 97 for the two, so they are not
// used.  8 tokens: 3 us, a call 7.5 us on the host.
template <typename W, typename T, int kN>
__global__ __launch_bounds__(kThreads) void embed_fwd_kernel(EmbedArgs p, int lanes) {
  constexpr int kAhead = 8;
  const int pieces = (p.dim + kN - 1) / kN, per = kThreads / lanes;
  const int at = threadIdx.x & (lanes - 1);
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int64_t row = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / lanes;
  if (row >= p.tokens) return;
  uint32_t next = key_of(p, row);
  for (; row < p.tokens; row += step) {
    const uint32_t key = next;
    if (row + step < p.tokens) next = key_of(p, row + step);
    const bool there = key < p.vocab;
    const W *from = static_cast<const W *>(p.weight) + (there ? key * p.w_stride : 0);
    T *to = static_cast<T *>(p.out) + row * p.dim;
    for (int q0 = at; q0 < pieces; q0 += kAhead * lanes) {
      Piece<W, kN> w[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        w[k].zero();
        if (there && q0 + k * lanes < pieces) load_piece(w[k], from, q0 + k * lanes, p.dim);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (q0 + k * lanes >= pieces) break;
        float v[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) v[e] = there ? w[k][e] * p.scale : 0.0f;
        store_piece<T, kN>(to, q0 + k * lanes, p.dim, v);
      }
    }
  }
}

// ------------------------------------------------------------------- sort --
// Pairs of id and token, a digit of up to kMaxBits bits a pass.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBits = 9, kBins = 1 << kMaxBits;
constexpr int kShort = 16384;       // most tokens of the short sort: one workgroup, in LDS
constexpr int kOwnTiles = 256;      // tiles up to which the scatter sums the counts itself

struct SortPass {
  const uint32_t *keys, *pos;  // null in the first pass: the ids themselves
  uint32_t *keys_out, *pos_out;
  uint32_t *counts;            // (tiles, bins): of each tile, or the places before it
  int64_t tiles;
  int shift, bits;
};

// Lanes of the wave whose digit is this lane's, among those in `in`.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, uint64_t in, int bits) {
#pragma unroll
  for (int b = 0; b < kMaxBits; ++b) {
    if (b < bits) {
      const bool bit = digit >> b & 1u;
      const uint64_t set = __ballot(bit);
      in &= bit ? set : ~set;
    }
  }
  return in;
}

// Rank of the lane's key among the wave's with the same digit so far, whose
// numbers are in `count`.
__device__ __forceinline__ uint32_t rank_of(uint32_t digit, bool in, int bits, uint32_t *count) {
  const int lane = threadIdx.x & 63;
  const uint64_t same = same_digit(digit, __ballot(in), bits);
  const int first = __ffsll(static_cast<unsigned long long>(same)) - 1;
  uint32_t old = 0u;
  if (in && lane == first)
    old = atomicAdd(&count[digit], static_cast<uint32_t>(__popcll(same)));
  old = __shfl(old, first < 0 ? 0 : first);
  return old + __popcll(same & ((uint64_t(1) << lane) - 1));
}

// Sum of v over the threads before this one, of kBins neighbouring threads
// that start at thread 0 (all threads of the workgroup call it).
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t *buf) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t up = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(up, d);
    if (lane >= d) up += o;
  }
  if (lane == 63) buf[wave] = up;
  __syncthreads();
  up -= v;
  for (int w = 0; w < wave; ++w) up += buf[w];
  __syncthreads();
  return up;
}

// Zeros in the rows row0 .. row1 - 1 of dweight whose bit in `there` (of row
// row0 on) is not set, by the whole workgroup.
template <typename W>
__device__ __forceinline__ void clear_rows(const EmbedArgs &p, int64_t row0, int64_t row1,
                                           const uint32_t *there) {
  constexpr int kN = 16 / sizeof(W);
  const int pieces = (p.dim + kN - 1) / kN, threads = blockDim.x;
  const int rows = static_cast<int>(row1 - row0), rs = threads / pieces, qs = threads % pieces;
  float zero[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) zero[e] = 0.0f;
  int r = threadIdx.x / pieces, q = threadIdx.x % pieces;
  while (r < rows) {
    if (!(there[r / 32] >> (r % 32) & 1u))
      store_piece<W, kN>(static_cast<W *>(p.dweight) + (row0 + r) * p.dim, q, p.dim, zero);
    r += rs;
    q += qs;
    if (q >= pieces) {
      q -= pieces;
      ++r;
    }
  }
}

// Zeros in the rows of ids that do not come, of the rows_per rows of one
// workgroup (of kSortThreads), which looks for them among all ids.
constexpr int kClearRows = 8192;  // rows it looks for at a time
template <typename W>
__device__ __forceinline__ void clear_group(const EmbedArgs &p, int64_t group, int64_t rows_per,
                                            uint32_t *there) {
  const int64_t begin = group * rows_per;
  const int64_t stop = begin + rows_per < p.vocab ? begin + rows_per : p.vocab;
  for (int64_t row0 = begin; row0 < stop; row0 += kClearRows) {
    const int64_t row1 = row0 + kClearRows < stop ? row0 + kClearRows : stop;
    for (int i = threadIdx.x; i < kClearRows / 32; i += kSortThreads) there[i] = 0u;
    __syncthreads();
    for (int t = threadIdx.x; t < p.tokens; t += kSortThreads) {
      const int64_t key = key_of(p, t);
      if (key >= row0 && key < row1)
        atomicOr(&there[(key - row0) / 32], 1u << ((key - row0) % 32));
    }
    __syncthreads();
    clear_rows<W>(p, row0, row1, there);
    __syncthreads();
  }
}

// The short sort, by workgroup 0; the others clear rows beside it.  Bound by the
// vector instructions that rank the keys on one CU (80 for a key and pass): 4096
// tokens of 32003 ids 14 us, 16384 41 us.  The clearing is bound by memory:
// 50000 rows of 2560 in fp32 but for those of 8192 tokens, 474 MB, 80 us (5.9
// TB/s).
template <typename W>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(EmbedArgs p, uint32_t *keys_out,
                                                                 uint32_t *pos_out, int passes,
                                                                 int bits, int64_t rows_per) {
  constexpr int kPer = kShort / kSortThreads;
  __shared__ uint32_t Key[kShort];
  __shared__ uint16_t Pos[kShort];
  __shared__ uint32_t Count[kSortWaves][kBins];
  __shared__ uint32_t Buf[kSortWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int n = static_cast<int>(p.tokens);
  if (blockIdx.x > 0) {
    clear_group<W>(p, blockIdx.x - 1, rows_per, Key);
    return;
  }
  // a wave holds neighbours, 64 at a time
  const int per = (n + kSortThreads - 1) / kSortThreads;
  uint32_t key[kPer], pos[kPer], rank[kPer];
  auto index = [&](int i) __attribute__((always_inline)) { return (wave * per + i) * 64 + lane; };
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < per) {
      pos[i] = index(i);
      key[i] = index(i) < n ? key_of(p, index(i)) : 0u;
    }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    const uint32_t mask = (1u << bits) - 1u;
    for (int i = tid; i < kSortWaves * kBins; i += kSortThreads) (&Count[0][0])[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per) rank[i] = rank_of(key[i] >> shift & mask, index(i) < n, bits, Count[wave]);
    __syncthreads();
    uint32_t sum = 0u;
    if (tid < kBins)
      for (int w = 0; w < kSortWaves; ++w) sum += Count[w][tid];
    uint32_t at = sum_before(tid < kBins ? sum : 0u, Buf);
    if (tid < kBins)
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = Count[w][tid];
        Count[w][tid] = at;
        at += c;
      }
    __syncthreads();
    const bool last = pass == passes - 1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per && index(i) < n) {
        const uint32_t to = Count[wave][key[i] >> shift & mask] + rank[i];
        if (last) {
          keys_out[to] = key[i];
          pos_out[to] = pos[i];
        } else {
          Key[to] = key[i];
          Pos[to] = static_cast<uint16_t>(pos[i]);
        }
      }
    if (last) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per && index(i) < n) {
        key[i] = Key[index(i)];
        pos[i] = Pos[index(i)];
      }
    __syncthreads();
  }
}

// The long sort: a tile of kPer keys a thread, a wave's 64 neighbours each.
template <int kPer>
__device__ __forceinline__ int64_t sort_index(int64_t tile, int i) {
  return tile * (kPer * kSortThreads) + (threadIdx.x >> 6) * (64 * kPer) + i * 64 +
         (threadIdx.x & 63);
}
__device__ __forceinline__ uint32_t sort_key(const EmbedArgs &p, const SortPass &s, int64_t at) {
  return s.keys ? s.keys[at] : key_of(p, at);
}

template <int kPer>
__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedArgs p, SortPass s) {
  __shared__ uint32_t Count[kBins];
  const uint32_t mask = (1u << s.bits) - 1u;
  for (int64_t tile = blockIdx.x; tile < s.tiles; tile += gridDim.x) {
    if (threadIdx.x < kBins) Count[threadIdx.x] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t at = sort_index<kPer>(tile, i);
      if (at < p.tokens) atomicAdd(&Count[sort_key(p, s, at) >> s.shift & mask], 1u);
    }
    __syncthreads();
    if (threadIdx.x < kBins) s.counts[tile * kBins + threadIdx.x] = Count[threadIdx.x];
    __syncthreads();
  }
}

// Places before each (tile, bin), in the order of the bins and in each that of
// the tiles.  Two threads have a bin, one the even tiles, one the odd ones; the
// first of them returns the sum.
constexpr int kHalves = kSortThreads / kBins;
__device__ __forceinline__ uint32_t places_before(const SortPass &s, int64_t tile,
                                                  uint32_t (*half)[kBins], uint32_t *buf) {
  const int bin = threadIdx.x % kBins, h = threadIdx.x / kBins;
  uint32_t before = 0u, all = 0u;
  for (int64_t t0 = h; t0 < s.tiles; t0 += 16 * kHalves) {
    uint32_t v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int64_t t = t0 + k * kHalves;
      v[k] = s.counts[(t < s.tiles ? t : t0) * kBins + bin];
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int64_t t = t0 + k * kHalves;
      before += t < tile ? v[k] : 0u;
      all += t < s.tiles ? v[k] : 0u;
    }
  }
  half[h][bin] = before;
  half[kHalves + h][bin] = all;
  __syncthreads();
  before = all = 0u;
  if (h == 0)
    for (int k = 0; k < kHalves; ++k) {
      before += half[k][bin];
      all += half[kHalves + k][bin];
    }
  return before + sum_before(all, buf);
}

// The same for more tiles, in place, by one workgroup in a launch of its own.
__global__ __launch_bounds__(kSortThreads) void embed_offsets_kernel(SortPass s) {
  __shared__ uint32_t Half[2 * kHalves][kBins];
  __shared__ uint32_t Buf[kSortWaves];
  uint32_t at = places_before(s, 0, Half, Buf);
  if (threadIdx.x >= kBins) return;
  uint32_t *count = s.counts + threadIdx.x;
  for (int64_t t0 = 0; t0 < s.tiles; t0 += 16) {
    uint32_t c[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) c[k] = t0 + k < s.tiles ? count[(t0 + k) * kBins] : 0u;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (t0 + k < s.tiles) count[(t0 + k) * kBins] = at;
      at += c[k];
    }
  }
}

// kOwn: the counts are those of each tile, and each workgroup forms the places
// of its own.  65536 tokens, 64 tiles: 8 us a pass, counting 5 us (3 us in the
// second pass), each bound by a handful of loads one after another.
template <int kPer, bool kOwn>
__global__ __launch_bounds__(kSortThreads) void embed_scatter_kernel(EmbedArgs p, SortPass s) {
  __shared__ uint32_t Count[kSortWaves][kBins];
  __shared__ uint32_t Half[2 * kHalves][kBins];
  __shared__ uint32_t Buf[kSortWaves];
  const int tid = threadIdx.x, wave = tid >> 6;
  const uint32_t mask = (1u << s.bits) - 1u;
  for (int64_t tile = blockIdx.x; tile < s.tiles; tile += gridDim.x) {
    uint32_t key[kPer], rank[kPer], pos[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t at = sort_index<kPer>(tile, i);
      key[i] = at < p.tokens ? sort_key(p, s, at) : 0u;
      pos[i] = s.pos && at < p.tokens ? s.pos[at] : static_cast<uint32_t>(at);
    }
    for (int i = tid; i < kSortWaves * kBins; i += kSortThreads) (&Count[0][0])[i] = 0u;
    uint32_t before = 0u;
    if constexpr (kOwn)
      before = places_before(s, tile, Half, Buf);
    else if (tid < kBins)
      before = s.counts[tile * kBins + tid];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      rank[i] = rank_of(key[i] >> s.shift & mask, sort_index<kPer>(tile, i) < p.tokens, s.bits,
                        Count[wave]);
    __syncthreads();
    if (tid < kBins) {
      // places of the tile's keys with this thread's digit, wave after wave
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = Count[w][tid];
        Count[w][tid] = before;
        before += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (sort_index<kPer>(tile, i) < p.tokens) {
        const uint32_t to = Count[wave][key[i] >> s.shift & mask] + rank[i];
        s.keys_out[to] = key[i];
        s.pos_out[to] = pos[i];
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

// Zeros in the rows of ids that do not come, from the sorted list: a workgroup
// (of kThreads) takes 32 rows a wave; lane l finds where id l of them begins.
constexpr int kSearchRows = 32 * kWavesPer;
template <typename W>
__device__ __forceinline__ void clear_sorted(const EmbedArgs &p, const uint32_t *keys, int64_t group,
                                             uint32_t *there) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = group * kSearchRows;
  const int64_t want = row0 + wave * 32 + (lane < 32 ? lane : 32);
  int64_t lo = 0, hi = p.tokens;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (keys[mid] < want)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int64_t next = __shfl_down(lo, 1);
  const uint64_t come = __ballot(lane < 32 && next > lo);
  if (lane == 0) there[wave] = static_cast<uint32_t>(come);
  __syncthreads();
  const int64_t row1 = row0 + kSearchRows < p.vocab ? row0 + kSearchRows : p.vocab;
  clear_rows<W>(p, row0, row1, there);
}

template <typename W>
__device__ __forceinline__ W *row_of(const EmbedArgs &p, uint32_t key) {
  return static_cast<W *>(p.dweight) + static_cast<int64_t>(key) * p.dim;
}
// old: what is there, 0 where the sum is written instead of added
template <typename W, int kN>
__device__ __forceinline__ void put_sum(const EmbedArgs &p, uint32_t key, int q,
                                        const float (&sum)[kN], const Piece<W, kN> &old) {
  float v[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) v[e] = fmaf(sum[e], p.scale, old[e]);
  store_piece<W, kN>(row_of<W>(p, key), q, p.dim, v);
}
// A wave takes one run and 64 pieces of the columns.  kAdd: the rows to add to
// are asked for together with those of dy.  The first `clears` workgroups, which
// wait for their searches, clear rows.  Bound by memory: 65536 tokens (5 in 61
// padding) of 768 columns, bf16 added to fp32, 42 us for 185 MB (4.4 TB/s); 8192
// of 2560, 28 us for 82 MB while the cleared rows drain from the last-level
// cache (20 us without).  Without the early request for the rows to add to: 49 us.
template <typename T, typename W, int kN, bool kAdd>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(EmbedArgs p, Runs r, uint32_t clears) {
  if constexpr (!kAdd) {
    __shared__ uint32_t There[kWavesPer];
    if (blockIdx.x < clears) {
      clear_sorted<W>(p, r.keys, blockIdx.x, There);
      return;
    }
  }
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pieces = (p.dim + kN - 1) / kN;
  const int cols = (pieces + 63) / 64;
  const uint32_t at = (blockIdx.x - clears) * kWavesPer + wave;
  const int64_t run = at / cols;
  if (run >= r.runs) return;
  const int q = static_cast<int>(at % cols) * 64 + lane;
  const int64_t from = run * r.len;
  const int n = static_cast<int>(p.tokens - from < r.len ? p.tokens - from : r.len);
  const int64_t mine = from + (lane < n ? lane : n - 1);
  const uint32_t key = r.keys[mine], pos = r.pos[mine];
  const uint32_t next = r.keys[mine + 1 < p.tokens ? mine + 1 : mine];
  // the first id may have begun in a run before
  bool came = from > 0 && r.keys[from > 0 ? from - 1 : 0] ==
                              static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(key));
  const uint64_t ends = __ballot(next != key || mine + 1 >= p.tokens);
  float acc[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) acc[e] = 0.0f;
  float *part = r.parts + run * 2 * r.row;
  const int safe = q < pieces ? q : pieces - 1;
  for (int j = 0; j < n; j += kAhead) {
    Piece<T, kN> dy[kAhead];
    Piece<W, kN> old[kAdd ? kAhead : 1];
    old[0].zero();
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int at = j + k < n ? j + k : n - 1;
      const int64_t t = static_cast<uint32_t>(__builtin_amdgcn_readlane(pos, at));
      load_piece(dy[k], static_cast<const T *>(p.dy) + t * p.dy_stride, safe, p.dim);
      if constexpr (kAdd) {
        const uint32_t id = __builtin_amdgcn_readlane(key, at);
        if (j + k < n && (ends >> at & 1) && id < p.vocab)
          load_piece(old[k], row_of<W>(p, id), safe, p.dim);
      }
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
          put_sum<W, kN>(p, id, q, acc, old[kAdd ? k : 0]);
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
// of that id, for 64 pieces of the columns: a wave by itself up to kAlone of
// them, more by the workgroup's waves together.  Four loads one after another
// (keys, the runs behind, partial rows): 10 us for the 65536 tokens above, 6 us
// for the 8192.
constexpr int kJoinWaves = 16, kAlone = 8;
template <typename W, int kN>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(EmbedArgs p, Runs r) {
  __shared__ float Sums[kJoinWaves][kN][64];
  __shared__ int64_t Behind[kJoinWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t run0 = static_cast<int64_t>(blockIdx.x) * kJoinWaves, run = run0 + wave;
  const int pieces = (p.dim + kN - 1) / kN;
  const int q = blockIdx.y * 64 + lane;
  float acc[kN];
  // the first partial row of the id that begins in a run, and every `step`-th
  // behind it
  Piece<W, kN> old;
  auto sum = [&](int64_t of, int64_t first, int64_t n, int64_t step) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < kN; ++e) acc[e] = 0.0f;
    const int at = q < pieces ? q : pieces - 1;
    const float *part = r.parts + (of + 1) * 2 * r.row;
    if (first == 0) get_piece<float, kN>(part - r.row, at, p.dim, acc);
    for (int64_t c = first; c < n; c += kAlone * step) {
      Piece<float, kN> v[kAlone];
#pragma unroll
      for (int k = 0; k < kAlone; ++k) {
        const int64_t row = c + k * step < n ? c + k * step : c;
        load_piece(v[k], part + row * 2 * r.row, at, p.dim);
      }
#pragma unroll
      for (int k = 0; k < kAlone; ++k)
#pragma unroll
        for (int e = 0; e < kN; ++e) acc[e] += c + k * step < n ? v[k][e] : 0.0f;
    }
  };
  // asks for the row that a sum is added to
  auto add_to = [&](uint32_t key) __attribute__((always_inline)) {
    old.zero();
    if (p.accumulate) load_piece(old, row_of<W>(p, key), q < pieces ? q : pieces - 1, p.dim);
  };
  const int64_t from = run * r.len, last = from + r.len - 1;
  int64_t behind = 0;
  if (last < p.tokens - 1) {
    const uint32_t key = r.keys[last], next = r.keys[last + 1], begin = r.keys[from];
    const uint32_t before = r.keys[from > 0 ? from - 1 : 0];
    if (key < p.vocab && next == key && !(from > 0 && begin == key && before == key)) {
      // the runs behind that begin with the id, 64 looked at at once
      for (;;) {
        const int64_t c = run + 1 + behind + lane;
        const bool on = c < r.runs && r.keys[c < r.runs ? c * r.len : 0] == key;
        const int more = __popcll(__ballot(on));
        behind += more;
        if (more < 64) break;
      }
      if (behind <= kAlone) {
        add_to(key);
        sum(run, 0, behind, 1);
        if (q < pieces) put_sum<W, kN>(p, key, q, acc, old);
        behind = 0;
      }
    }
  }
  if (lane == 0) Behind[wave] = behind;
  __syncthreads();
  for (int w = 0; w < kJoinWaves; ++w) {
    const int64_t n = Behind[w];
    if (n == 0) continue;
    const uint32_t key = r.keys[(run0 + w + 1) * r.len - 1];
    if (wave == 0) add_to(key);
    sum(run0 + w, wave, n, kJoinWaves);
#pragma unroll
    for (int e = 0; e < kN; ++e) Sums[wave][e][lane] = acc[e];
    __syncthreads();
    if (wave == 0 && q < pieces) {
      for (int k = 1; k < kJoinWaves; ++k)
#pragma unroll
        for (int e = 0; e < kN; ++e) acc[e] += Sums[k][e][lane];
      put_sum<W, kN>(p, key, q, acc, old);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- few tokens --
// Up to kFew tokens in one launch, without a sort: a wave takes a token and 64
// pieces of the columns, finds the tokens of the same id among all ids, and sums
// their rows if its own is the first of them.  Workgroups behind the first
// `sums` clear rows.  64 tokens 7 us, 256 of 768 columns 8 us (sorted, in three
// launches, 18 us); a row that all 256 tokens have is summed by one wave for
// each 64 pieces.
constexpr int kFew = 256;
template <typename T, typename W, int kN>
__global__ __launch_bounds__(kSortThreads) void embed_few_kernel(EmbedArgs p, uint32_t sums,
                                                                int64_t rows_per) {
  __shared__ uint32_t There[kClearRows / 32];
  if (blockIdx.x >= sums) {
    clear_group<W>(p, blockIdx.x - sums, rows_per, There);
    return;
  }
  constexpr int kAhead = 8, kWords = kFew / 64;
  const int lane = threadIdx.x & 63, n = static_cast<int>(p.tokens);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pieces = (p.dim + kN - 1) / kN, cols = (pieces + 63) / 64;
  const uint32_t task = blockIdx.x * kSortWaves + wave;
  const int own = task / cols;
  if (own >= n) return;
  const int q = static_cast<int>(task % cols) * 64 + lane, safe = q < pieces ? q : pieces - 1;
  uint32_t keys[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) keys[w] = key_of(p, w * 64 + lane < n ? w * 64 + lane : 0);
  const uint32_t key = __builtin_amdgcn_readfirstlane(key_of(p, own));
  if (key >= p.vocab) return;
  uint64_t same[kWords];
  int count = 0;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    same[w] = __ballot(w * 64 + lane < n && keys[w] == key);
    count += __popcll(same[w]);
  }
  // the first of them
  bool earlier = false;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const int bits = own - w * 64;
    if (bits > 0) earlier |= (bits >= 64 ? same[w] : same[w] & ((uint64_t(1) << bits) - 1)) != 0;
  }
  if (earlier) return;
  Piece<W, kN> old;
  old.zero();
  if (p.accumulate) load_piece(old, row_of<W>(p, key), safe, p.dim);
  float acc[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) acc[e] = 0.0f;
  int t = 0;
  // the next of them, or the last one again (no indexing by a variable, which
  // would put the masks into memory)
  auto next = [&]() __attribute__((always_inline)) {
    bool found = false;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const bool here = !found && same[w] != 0;
      t = here ? w * 64 + __ffsll(static_cast<unsigned long long>(same[w])) - 1 : t;
      same[w] &= here ? same[w] - 1 : ~uint64_t(0);
      found |= here;
    }
  };
  for (int j = 0; j < count; j += kAhead) {
    Piece<T, kN> dy[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      next();
      load_piece(dy[k], static_cast<const T *>(p.dy) + t * p.dy_stride, safe, p.dim);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int e = 0; e < kN; ++e) acc[e] += j + k < count ? dy[k][e] : 0.0f;
  }
  if (q < pieces) put_sum<W, kN>(p, key, q, acc, old);
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Columns of a lane in the sums.
constexpr int kSumPiece = 4;

// Sorted tokens a run has: short ones where there are few waves, each of which
// waits for its rows in turn, long ones where partial rows would be many.
// (Added to a gradient, runs of 8, 16 and 32: 8192 tokens of 768 columns 35, 36
// and 41 us, 16384 of 768 42, 39 and 43 us, 16384 of 2560 92, 84 and 80 us.)
int run_len(int64_t tokens, int64_t cols) {
  return tokens * cols < 32768 ? 8 : tokens * cols < 65536 ? 16 : 32;
}

// One workgroup sorts 4096, 8192 and 16384 tokens in 14, 22 and 41 us, the
// launches of the long sort take 24 us; but beside the short one rows are
// cleared.  (8192 tokens of 768 columns, short and long: added 40 and 35 us, as
// a new gradient of 32000 rows 43 and 51 us; 16384 of 2560, a new one of 50000
// rows, 512 MB, 147 and 160 us, of 768 and 32000 rows, 98 MB, 68 and 57 us.)
bool sort_is_short(const EmbedArgs &a, int64_t row_bytes) {
  if (a.tokens <= 4096) return true;
  if (a.accumulate || a.tokens > kShort) return false;
  return a.tokens <= 8192 || a.vocab * row_bytes >= int64_t(256) << 20;
}

// Workspace: two lists of keys and positions, the counts, the partial rows.
struct Layout {
  int64_t tiles, runs, row;
  int len, per;  // sorted tokens a run has; keys a thread of the long sort has
  int64_t keys[2], pos[2], counts, parts, bytes;
};
Layout layout_of(int64_t tokens, int64_t dim) {
  Layout l;
  l.per = tokens <= kOwnTiles / 2 * kSortThreads ? 1 : 4;
  l.tiles = (tokens + l.per * kSortThreads - 1) / (l.per * kSortThreads);
  l.len = run_len(tokens, (dim + 64 * kSumPiece - 1) / (64 * kSumPiece));
  l.runs = (tokens + l.len - 1) / l.len;
  l.row = up(dim, 4);
  const int lists = 2;
  int64_t at = 0;
  for (int i = 0; i < lists; ++i) {
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

// Passes and bits a pass for keys 0..vocab.
void digits_of(int64_t vocab, int &passes, int &bits) {
  int all = 1;
  while (vocab >> all) ++all;
  passes = (all + kMaxBits - 1) / kMaxBits;
  bits = (all + passes - 1) / passes;
}

template <typename T, typename W>
int launch_bwd(const EmbedArgs &a, hipStream_t s) {
  constexpr int kN = kSumPiece;
  const unsigned cols = static_cast<unsigned>(((a.dim + kN - 1) / kN + 63) / 64);
  // workgroups that clear rows, and the rows of each, beside few tokens or the
  // short sort
  const unsigned clears = a.accumulate ? 0u : static_cast<unsigned>(a.vocab < 255 ? a.vocab : 255);
  const int64_t rows_per = a.accumulate ? 1 : (a.vocab + clears - 1) / clears;
  if (a.tokens <= kFew) {
    const unsigned sums = static_cast<unsigned>((a.tokens * cols + kSortWaves - 1) / kSortWaves);
    if (sums + clears == 0) return 0;
    hipLaunchKernelGGL((embed_few_kernel<T, W, kN>), dim3(sums + clears), dim3(kSortThreads), 0, s,
                       a, sums, rows_per);
    return static_cast<int>(hipGetLastError());
  }
  const Layout l = layout_of(a.tokens, a.dim);
  char *ws = static_cast<char *>(a.workspace);
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t *>(ws + at); };
  int passes, bits, to = 0;
  digits_of(a.vocab, passes, bits);
  const bool brief = sort_is_short(a, a.dim * static_cast<int64_t>(sizeof(W)));
  if (brief) {
    hipLaunchKernelGGL(embed_sort_kernel<W>, dim3(1 + clears), dim3(kSortThreads), 0, s, a,
                       words(l.keys[0]), words(l.pos[0]), passes, bits, rows_per);
  } else {
    SortPass sort{nullptr, nullptr, nullptr, nullptr, words(l.counts), l.tiles, 0, bits};
    const unsigned grid = static_cast<unsigned>(l.tiles < 65536 ? l.tiles : 65536);
    for (int pass = 0; pass < passes; ++pass) {
      sort.shift = pass * bits;
      sort.keys_out = words(l.keys[to]);
      sort.pos_out = words(l.pos[to]);
      auto go = [&](auto kernel, unsigned groups) {
        hipLaunchKernelGGL(kernel, dim3(groups), dim3(kSortThreads), 0, s, a, sort);
      };
      if (l.per == 1) {
        go(embed_count_kernel<1>, grid);
        go(embed_scatter_kernel<1, true>, grid);
      } else if (l.tiles <= kOwnTiles) {
        go(embed_count_kernel<4>, grid);
        go(embed_scatter_kernel<4, true>, grid);
      } else {
        go(embed_count_kernel<4>, grid);
        hipLaunchKernelGGL(embed_offsets_kernel, dim3(1), dim3(kSortThreads), 0, s, sort);
        go(embed_scatter_kernel<4, false>, grid);
      }
      sort.keys = sort.keys_out;
      sort.pos = sort.pos_out;
      to ^= 1;
    }
    to ^= 1;
  }
  const Runs r{words(l.keys[to]), words(l.pos[to]), reinterpret_cast<float *>(ws + l.parts), l.runs,
               l.row, l.len};
  const unsigned sums = static_cast<unsigned>((l.runs * cols + kWavesPer - 1) / kWavesPer);
  const unsigned searches =
      a.accumulate || brief ? 0u
                            : static_cast<unsigned>((a.vocab + kSearchRows - 1) / kSearchRows);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(searches + sums), dim3(kThreads), 0, s, a, r, searches);
  };
  if (a.accumulate)
    go(embed_sum_kernel<T, W, kN, true>);
  else
    go(embed_sum_kernel<T, W, kN, false>);
  if (l.runs > 1)
    hipLaunchKernelGGL((embed_join_kernel<W, kN>),
                       dim3(static_cast<unsigned>((l.runs + kJoinWaves - 1) / kJoinWaves), cols),
                       dim3(64 * kJoinWaves), 0, s, a, r);
  return static_cast<int>(hipGetLastError());
}

template <typename W, typename T, int kN>
int launch_fwd(const EmbedArgs &a, hipStream_t s) {
  const int pieces = (a.dim + kN - 1) / kN;
  int lanes = 8;
  while (lanes < 64 && lanes < pieces) lanes *= 2;
  const int64_t per = kThreads / lanes, groups = (a.tokens + per - 1) / per;
  const int64_t most = 4096;
  hipLaunchKernelGGL((embed_fwd_kernel<W, T, kN>),
                     dim3(static_cast<unsigned>(groups < most ? groups : most)), dim3(kThreads), 0,
                     s, a, lanes);
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int64_t embed_bwd_workspace(int64_t tokens, int64_t dim) {
  return tokens <= kFew ? 0 : layout_of(tokens, dim).bytes;
}

int launch_embed_fwd(const EmbedArgs &a, bool w_bf16, bool bf16, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (w_bf16)
    return bf16 ? launch_fwd<uint16_t, uint16_t, 8>(a, s) : launch_fwd<uint16_t, float, 4>(a, s);
  return bf16 ? launch_fwd<float, uint16_t, 8>(a, s) : launch_fwd<float, float, 4>(a, s);
}

int launch_embed_bwd(const EmbedArgs &a, bool w_bf16, bool bf16, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (bf16)
    return w_bf16 ? launch_bwd<uint16_t, uint16_t>(a, s) : launch_bwd<uint16_t, float>(a, s);
  return w_bf16 ? launch_bwd<float, uint16_t>(a, s) : launch_bwd<float, float>(a, s);
}

}  // namespace ssm
