// ssm_linattn_internal.h -- launch interface between the linear-attention entry points
// (ssm_linattn_api.cpp) and their gfx950 kernels.  Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ssm {

// Tokens per chunk: what one pass of the matrix-core kernels takes at once.
constexpr int kLinChunkBf16 = 64;
constexpr int kLinChunkF32 = 32;
constexpr int kLinMaxDim = 256;     // largest query/key and value head size
constexpr int kLinDecayNone = 0, kLinDecayToken = 1, kLinDecayHead = 2;

// How the token rows are cut.  Every sequence is cut into segments of
// seg_len tokens (a multiple of the chunk) from its own start; a segment has
// a slot.  Equal sequences: slot = seq * segs + seg.  Packed ones (cu): slot
// = cu[seq] / seg_len + seq + seg, which leaves gaps but never overlaps.
struct LinPlan {
  const int32_t *cu;    // (nseq + 1) row offsets on the device, or null
  int64_t tokens;       // rows of the token arrays
  int64_t seqlen;       // equal sequences: rows of each
  int64_t seg_len;
  int64_t segs;         // equal sequences: segments of each
  int64_t slots;        // segments over all sequences (upper bound if packed)
  int nseq, heads;
  int vec;              // every row piece of 16 bytes may be moved whole
};

// One (tokens, heads, d) operand.
struct LinSide {
  const void *p;
  int64_t stride;       // elements between token rows
  int d;                // elements of a head
  int div;              // value heads per head of this operand
};

// One pass over the chunks of every segment (ssm_linattn_core.h):
//   out_t = inter * w_t (sum_a q_t[a] S[a][:]) + inside * sum_s m_ts (q_t . k_s) v_s
//   S    <- decay S + into * sum_s w'_s k_s v_s^T
// in token order, or against it.
struct LinCore {
  LinPlan plan;
  LinSide q, k, v;
  const float *g;
  int g_kind;
  float inter, inside, into;
  // state entering each segment, element (a, b) at a * sa + b * sb: in_slots
  // by (slot, head), else in_seqs by (sequence, head), else zero
  const float *in_slots, *in_seqs;
  // state leaving: of every segment by slot (state pass), and of each
  // sequence's last segment (first, against token order); kLinOutDot in
  // token order: instead the state before each sequence's last chunk
  float *out_slots, *out_seqs;
  float *out_decay;     // state pass: exp of each segment's sum of decays (slot, head)
  int sa, sb;
  void *out;            // (tokens, heads, v.d), or null (state pass)
  int out_f32;          // out in fp32 whatever the activations
  // kLinOutDot: the state part's dot products with the rows of x, dots (slice,
  // tokens, heads)
  LinSide x;
  float *dots;
};

enum LinMode { kLinState = 0, kLinOut = 1, kLinOutDot = 2 };

struct LinChain {       // running states of the segments, in place
  LinPlan plan;
  float *states;        // (slot, head, size): what each adds -> what enters it
  const float *decay;   // (slot, head)
  const float *first;   // (sequence, head, size) or null: zero
  int64_t size;
  int reverse;
};

struct LinPairs {       // sums over token pairs inside each chunk
  LinPlan plan;         // its segments are the chunks
  LinSide q, k, v, o;
  const float *g;
  int g_kind;
  float scale;
  float *out;           // (tokens, heads)
};

struct LinDecayGrad {
  LinPlan plan;
  const float *pairs, *xdots, *ydots;  // (tokens, heads); dots by slice
  int slices;                          // of the dots: 1 or 2
  const float *states, *adjoints;      // entering each segment, by slot
  // (sequence, head, size): the state before the last chunk, the adjoint of
  // the final state (null: zero)
  const float *last, *dlast;
  int size;
  const float *g;
  int g_kind, chunk;
  float *dg;
};

struct LinZero {          // rows outside the sequences, set to 0
  LinPlan plan;
  struct { void *p; int64_t row_bytes; } arrays[4];  // those with p first
};

struct LinStep {
  float *state;
  const void *q, *k, *v;
  const float *g;
  int g_kind;
  const int32_t *slot_of;  // or null
  void *o;
  float scale;
  int64_t batch, slots, q_stride, k_stride, v_stride;
  int heads, qk_heads, dk, dv;
};

// tokens of a chunk, output columns of one workgroup
int linattn_chunk(bool bf16);
int linattn_slice(int dv);
// whether a workgroup takes two value heads: they share the first two
// operands (`div` value heads to one of theirs) and have at most 64 columns
bool linattn_pairs_heads(int div, int dv);
int launch_linattn_out_bf16(const LinCore &a, void *stream);
int launch_linattn_out_f32(const LinCore &a, void *stream);
// the states that segments add (a: in token order; back, if not null: against it)
int launch_linattn_states_bf16(const LinCore &a, const LinCore *back, void *stream);
int launch_linattn_states_f32(const LinCore &a, const LinCore *back, void *stream);
// dq, dk, dv and, if not null, the sums over pairs
int launch_linattn_grads_bf16(const LinCore &dq, const LinCore &dk, const LinCore &dv,
                              const LinPairs *pairs, void *stream);
int launch_linattn_grads_f32(const LinCore &dq, const LinCore &dk, const LinCore &dv,
                             const LinPairs *pairs, void *stream);
// one or two (b not null) chains over the same segments
int launch_linattn_chain(const LinChain &a, const LinChain *b, void *stream);
int launch_linattn_decay_grad(const LinDecayGrad &a, void *stream);
// sums of `div` consecutive heads, for two arrays: in (tokens, heads, d) fp32 -> out
// (tokens, heads / div, d)
int launch_linattn_head_sum(const float *in0, const float *in1, void *out0, void *out1,
                            const LinPlan &plan, int div, int d, bool bf16, void *stream);
// out[h] = sum of in[t][h]
int launch_linattn_token_sum(const float *in, float *out, const LinPlan &plan, void *stream);
int launch_linattn_zero_outside(const LinZero &a, void *stream);
int launch_linattn_step(const LinStep &a, bool bf16, void *stream);

}  // namespace ssm
