/*
 * ssm_linattn.h -- C ABI of linear attention with a decay for each head, and
 * of the block norm that surrounds a layer's mixer, on MI355X (gfx950).
 *
 * Linear attention keeps, per sequence and value head, a matrix state in
 * place of a cache of keys and values:
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T       (qk_dim x v_dim)
 *   o_t = scale * S_t^T q_t
 * g is a log decay: one a token and head (gated forms; the SSD form of
 * Mamba-2 with q = C, k = B, v = dt x, g = dt A), one a head, or none.
 * ssm_ssd_fwd (ssm_scan.h) computes that SSD form from channel-major rows with
 * softplus, D and the gate inside, forward only; its states are (headdim,
 * dstate), the transpose of those here.
 *
 * Conventions are those of ssm_scan.h (device pointers owned by the caller,
 * nothing allocated, work enqueued on `stream`, statuses, ssm_last_error(),
 * every argument checked before the first HIP call), except for the layout,
 * which is that of the projections before and after the mixer: token rows,
 * each row head after head, the head's elements fastest.
 *   q, k        (tokens, qk_heads, qk_dim)   rows q_stride, k_stride elements apart
 *   v           (tokens, heads, v_dim)       rows v_stride elements apart
 *   o           (tokens, heads, v_dim)       dense
 *   g           (tokens, heads) fp32 dense, or (heads) fp32, or NULL
 *   states      (sequences, heads, qk_dim, v_dim) fp32 dense
 * Value head h uses query/key head h / (heads / qk_heads).  A row stride
 * larger than the row lets q, k and v be parts of one projection's output.
 * Sizes: qk_dim and v_dim 1..256; heads a multiple of qk_heads; row strides
 * up to 2^22; activations fp32 or bf16 (ssm_dtype).  Rows whose starts,
 * strides and head sizes are multiples of 16 bytes are read 16 bytes at a
 * time; others element by element.  Calls that would need a launch of 2^32
 * threads are refused (SSM_ERR_UNSUPPORTED, by ssm_linattn_plan too): segments
 * (below) times heads times the 128-column slices of the outputs, and with dg
 * chunks times heads as well, have to stay under 2^23.
 *
 * Sequences: without cu_seqlens the tokens are nseq sequences of tokens /
 * nseq rows; with it (device, int32, nseq + 1 offsets, not falling, within
 * 0..tokens) sequence i is rows cu_seqlens[i] .. cu_seqlens[i + 1] - 1, of
 * any length, 0 included.  Rows before the first and behind the last
 * sequence are not read, and written only with SSM_FLAG_ZERO_OUTSIDE.  The
 * offsets are not checked (that would need a synchronisation): ones outside
 * 0..tokens are brought into that range and a falling one ends its sequence, so
 * that no memory outside the arrays is touched, but results are then
 * unspecified.
 */
#ifndef SSM_LINATTN_H
#define SSM_LINATTN_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* g holds one log decay a head, for every token: (heads) */
#define SSM_FLAG_HEAD_DECAY 8u
/* rows of o, dq, dk, dv and dg that lie in no sequence are set to 0 (without
 * it they are left as they are) */
#define SSM_FLAG_ZERO_OUTSIDE 32u

/* How ssm_linattn_fwd (backward = 0) or ssm_linattn_bwd (backward = 1, or 2
 * with dg) cuts the sequences, in plan_out[4] (no HIP call):
 *  [0] tokens per segment: segments are taken in parallel, each from the
 *      state that a pass over the segments before it formed
 *  [1] segments (an upper bound with cu_seqlens)
 *  [2] tokens per chunk of the matrix products
 *  [3] 1 if that pass is made, 0 if every sequence is one segment
 * packed: nonzero with cu_seqlens. */
int ssm_linattn_plan(int64_t tokens, int64_t nseq, int packed, int64_t heads, int64_t qk_heads,
                     int64_t qk_dim, int64_t v_dim, int dtype, int backward, int64_t *plan_out);

/* Bytes of device workspace for ssm_linattn_fwd (0 where every sequence is
 * one segment). */
int ssm_linattn_workspace_size(int64_t tokens, int64_t nseq, int packed, int64_t heads,
                               int64_t qk_heads, int64_t qk_dim, int64_t v_dim, int dtype,
                               size_t *bytes);

/* Linear attention over whole sequences (prompts, training).
 *  q, k, v     required, activation dtype; may overlap each other
 *  g           nullable fp32; (tokens, heads), or (heads) with
 *              SSM_FLAG_HEAD_DECAY.  Natural logarithm; -inf forgets all that
 *              came before the token; above 0 the state grows, and sums of g
 *              over runs of tokens have to stay below 88 (e^88 is near the
 *              end of fp32's range)
 *  scale       factor of o
 *  h0          nullable fp32: state before each sequence (zero if NULL)
 *  cu_seqlens  nullable (see above)
 *  o           required output, activation dtype, dense; overlaps no input
 *  h_final     nullable fp32 output: state after each sequence (an empty one
 *              hands h0 on); overlaps no input
 *  tokens >= 0, nseq >= 1, tokens below 2^31
 *  workspace   >= ssm_linattn_workspace_size() bytes, 256-byte aligned, in
 *              use until the enqueued work is done; its contents on entry do
 *              not matter
 * bf16: the weighted products of token pairs, and the state where o is read
 * from it, are rounded to bf16 once; what enters the state does so with 24
 * bits (as three bf16 values) and is carried in fp32.  fp32 runs in fp32.
 * An infinity or NaN in a token's q, k, v or g reaches the results that the
 * recurrence lets it reach (no token before it, no other column than its own
 * if it is in v), but may be NaN there where the recurrence has an infinity. */
int ssm_linattn_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const float *g, unsigned flags, float scale,
                    const float *h0, const int32_t *cu_seqlens, void *o, float *h_final,
                    int64_t tokens, int64_t nseq, int64_t heads, int64_t qk_heads, int64_t qk_dim,
                    int64_t v_dim, int dtype, void *workspace, size_t workspace_bytes,
                    void *stream);

/* Bytes of device workspace for ssm_linattn_bwd.  want_dg: 0 without dg, 1
 * with dg of a decay a token, 2 with dg of a decay a head. */
int ssm_linattn_bwd_workspace_size(int64_t tokens, int64_t nseq, int packed, int64_t heads,
                                   int64_t qk_heads, int64_t qk_dim, int64_t v_dim, int dtype,
                                   int want_dg, size_t *bytes);

/* Gradients of ssm_linattn_fwd for a loss with gradient d_o (dense, as o)
 * with respect to o and dh_final (nullable: zero) with respect to h_final.
 * With M_t the adjoint of S_t:
 *   M_t = exp(g_{t+1}) M_{t+1} + scale q_t do_t^T   (after the last: dh_final)
 *   dq_t = scale S_t do_t,   dk_t = M_t v_t,   dv_t = M_t^T k_t,
 *   dg_t = exp(g_t) <M_t, S_{t-1}>,   dh0 = exp(g_0) M_0
 * summed over the value heads that share a query/key head (dq, dk) and, for
 * a decay a head, over all tokens (dg).
 *  dq, dk      required outputs, activation dtype, dense (tokens, qk_heads, qk_dim)
 *  dv          required output, activation dtype, dense (tokens, heads, v_dim)
 *  dg          nullable output, fp32, shape of g; only with g
 *  dh0         nullable output, fp32
 *  workspace   >= ssm_linattn_bwd_workspace_size() bytes, 256-byte aligned
 * Roundings as in the forward pass, except that with dg the state and its
 * adjoint enter dq and dk, as well as dg, with 24 bits instead of bf16's 8.
 * An infinity or NaN in a token's q, k, v or d_o reaches dq of no token before
 * it and dk and dv of none behind it; dg of its whole sequence, and with a NaN
 * in g dk and dv of the chunk around it, may be NaN.
 * Sums run in a fixed order: the same call gives the same bits. */
int ssm_linattn_bwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const float *g, unsigned flags, float scale,
                    const float *h0, const int32_t *cu_seqlens, const void *d_o,
                    const float *dh_final, void *dq, void *dk, void *dv, float *dg, float *dh0,
                    int64_t tokens, int64_t nseq, int64_t heads, int64_t qk_heads, int64_t qk_dim,
                    int64_t v_dim, int dtype, void *workspace, size_t workspace_bytes,
                    void *stream);

/* One token of `batch` sequences on states kept in slots (decoding).
 *  state       required fp32 (nslots, heads, qk_dim, v_dim): read, advanced,
 *              written back
 *  q, k, v     required, activation dtype: batch rows, strides as above
 *  g           nullable fp32: (batch, heads), or (heads) with SSM_FLAG_HEAD_DECAY
 *  slots       nullable int32 (batch), device: the slot of each row; NULL:
 *              row b has slot b (batch <= nslots).  A row whose slot is out of
 *              0..nslots-1, or already an earlier row's, touches no state and
 *              its o is 0 (idle rows of a batch: -1)
 *  o           required output, activation dtype, dense (batch, heads, v_dim)
 *  batch >= 0
 * Arithmetic is fp32.  Steps over tokens 0..L-1 give ssm_linattn_fwd's o and
 * h_final up to rounding. */
int ssm_linattn_step(float *state, const void *q, int64_t q_stride, const void *k,
                     int64_t k_stride, const void *v, int64_t v_stride, const float *g,
                     unsigned flags, float scale, const int32_t *slots, void *o, int64_t batch,
                     int64_t nslots, int64_t heads, int64_t qk_heads, int64_t qk_dim,
                     int64_t v_dim, int dtype, void *stream);

/* The norms on both sides of a block's end, with its gate and its residual
 * scale, in one pass over the rows.  With `groups` equal parts of a row:
 *   n = x / sqrt(mean_part(x^2) + eps) * w_post     (without w_post: n = x)
 *   r = residual + n * silu(z) * scale              (each factor, and the
 *                                                    residual, optional)
 *   y = r / sqrt(mean_row(r^2) + eps) * w_pre       (only with w_pre)
 * x is the mixer's output: with groups = heads this is the norm of each head
 * gated by silu(z) that follows linear attention; with a residual, the sum
 * that ends a block and the norm that begins the next.
 *  x            required, activation dtype (rows, dim), rows x_stride apart
 *  w_post       nullable fp32 (dim);  groups divides dim, 1 without w_post
 *  z            nullable, activation dtype (rows, dim), rows z_stride apart
 *  scale        nullable fp32 (dim)
 *  residual     nullable (rows, dim), rows residual_stride apart
 *  w_pre        nullable fp32 (dim)
 *  r            nullable output (rows, dim) dense (required without w_pre)
 *  y            output, activation dtype (rows, dim) dense; required with
 *               w_pre, NULL without
 *  dtype        activations;  residual_dtype: residual and r (the
 *               activations' or SSM_DTYPE_F32)
 *  0 <= rows < 2^22; dim 1..16384, at most 8192 with groups > 1; eps > 0
 * With z and w_pre but no w_post, y is the norm of the gated row, x silu(z),
 * as Mamba-2 has it.  Squares are summed in fp32: their mean has to lie within
 * its range (elements up to about 1e17).
 * y is formed from r before r is rounded.  Outputs may not overlap inputs,
 * except that r may be exactly the residual, in place (dense rows). */
int ssm_block_norm_fwd(const void *x, int64_t x_stride, const float *w_post, const void *z,
                       int64_t z_stride, const float *scale, const void *residual,
                       int64_t residual_stride, const float *w_pre, void *r, void *y,
                       int64_t rows, int64_t dim, int64_t groups, float eps, int dtype,
                       int residual_dtype, void *stream);

/* Bytes of device workspace for ssm_block_norm_bwd: partial sums of the
 * weights' gradients. */
int ssm_block_norm_bwd_workspace_size(int64_t rows, int64_t dim, size_t *bytes);

/* Gradients of ssm_block_norm_fwd, from its inputs (r and y are formed
 * again), for gradients dr of r (residual_dtype) and dy of y (activation
 * dtype); dr nullable (zero), dy required with w_pre and NULL without.  Both
 * dense.
 *  dx                      required, activation dtype, dense
 *  dw_post, dscale, dw_pre nullable fp32 (dim), each only with its input
 *  dz                      nullable, activation dtype, dense; only with z
 *  dresidual               nullable, residual_dtype, dense; only with residual
 *  workspace               >= ssm_block_norm_bwd_workspace_size() bytes,
 *                          256-byte aligned
 * Sums over rows run in a fixed order.  Outputs overlap nothing. */
int ssm_block_norm_bwd(const void *x, int64_t x_stride, const float *w_post, const void *z,
                       int64_t z_stride, const float *scale, const void *residual,
                       int64_t residual_stride, const float *w_pre, const void *dr,
                       const void *dy, void *dx, float *dw_post, void *dz, float *dscale,
                       void *dresidual, float *dw_pre, int64_t rows, int64_t dim, int64_t groups,
                       float eps, int dtype, int residual_dtype, void *workspace,
                       size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SSM_LINATTN_H */
