/*
 * ssm_model.h -- C ABI of what stands around a model's blocks on MI355X
 * (gfx950): the embedding, the layer norm, their gradients, and the global
 * norm of all gradients with their clipping.
 *
 * Conventions are those of ssm_scan.h (device pointers owned by the caller,
 * nothing allocated, work enqueued on `stream`, statuses, ssm_last_error(),
 * every argument checked before the first HIP call).  Rows are token-major,
 * as in ssm_linattn.h: (rows, dim), the elements of a row dense, rows
 * `*_stride` elements apart where a stride is given (dim .. 2^22), dense
 * elsewhere.  Activations are fp32 or bf16 (ssm_dtype), each array with a
 * type of its own where the call takes several.  Any row start and any dim
 * are read in pieces of up to 16 bytes; arrays need the alignment of their
 * elements only.  Arithmetic is fp32, sums run in a fixed order (the same
 * call gives the same bits), each output is rounded once.
 * An infinity or NaN stays in the rows, columns and sums that its formula
 * gives it to.
 */
#ifndef SSM_MODEL_H
#define SSM_MODEL_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* types of ids */
typedef enum {
    SSM_INDEX_I32 = 0,
    SSM_INDEX_I64 = 1
} ssm_index;

/* ssm_embed_bwd: dweight is added to (rows whose id does not come are not
 * touched) instead of written as a whole */
#define SSM_FLAG_ACCUMULATE 64u

/* ------------------------------------------------------------ embedding --
 * out_t = scale * weight[ids_t].  An id outside 0..vocab-1 (padding: -1) gives
 * a row of zeros and has no gradient.
 *  ids      required (tokens), int32 or int64 (ssm_index), device
 *  weight   required (vocab, dim), weight_dtype, rows weight_stride apart
 *  out      required output (tokens, dim) dense, dtype; overlaps no input
 *  0 <= tokens < 2^28, 1 <= vocab < 2^30, 1 <= dim <= 65536, tokens * dim below
 *  2^38 - 1024 */
int ssm_embed_fwd(const void *ids, const void *weight, int64_t weight_stride, void *out,
                  int64_t tokens, int64_t vocab, int64_t dim, float scale, int index_type,
                  int weight_dtype, int dtype, void *stream);

/* Bytes of device workspace for ssm_embed_bwd.  vocab is checked; the size does
 * not depend on it in this build. */
int ssm_embed_bwd_workspace_size(int64_t tokens, int64_t vocab, int64_t dim, size_t *bytes);

/* The gradient of the weight: dweight_v = scale * sum of dy_t over the tokens t
 * with ids_t = v, in fp32, in the order of the tokens, cut into runs whose
 * length and borders follow from the sizes and the ids; with
 * SSM_FLAG_ACCUMULATE that sum is added to dweight_v before the rounding.
 *  dy         required (tokens, dim), dtype, rows dy_stride apart
 *  dweight    required output (vocab, dim) dense, weight_dtype; every row is
 *             written (0 where no token has the id) unless it is added to;
 *             overlaps no input
 *  workspace  >= ssm_embed_bwd_workspace_size() bytes, 256-byte aligned, in use
 *             until the enqueued work is done; its contents on entry do not
 *             matter
 * Sizes as in ssm_embed_fwd. */
int ssm_embed_bwd(const void *ids, const void *dy, int64_t dy_stride, void *dweight,
                  int64_t tokens, int64_t vocab, int64_t dim, float scale, unsigned flags,
                  int index_type, int dtype, int weight_dtype, void *workspace,
                  size_t workspace_bytes, void *stream);

/* ----------------------------------------------------------- layer norm --
 * The residual sum and the norm after it, per row:
 *   r = x + residual                       (without a residual: r = x)
 *   y = (r - mean(r)) / sqrt(var(r) + eps) * weight + bias
 * with var the mean of the squared differences from the mean, formed from the
 * differences themselves.  y is formed from r before r is rounded.  Where the
 * squares pass fp32's largest number (differences over about 1.8e19) the variance
 * is infinite, and y the bias.
 * (ssm_block_norm_fwd, ssm_linattn.h, has the norm without mean and bias.)
 *  x         required, x_dtype (rows, dim), rows x_stride apart
 *  residual  nullable, residual_dtype (rows, dim), rows residual_stride apart
 *  weight    nullable fp32 (dim)
 *  bias      nullable fp32 (dim)
 *  r         nullable output, residual_dtype (rows, dim) dense; NULL without a
 *            residual
 *  y         required output, dtype (rows, dim) dense
 *  types     x_dtype bf16: dtype bf16, residual_dtype either; x_dtype fp32:
 *            residual_dtype fp32, dtype either.  residual_dtype is x_dtype
 *            without a residual
 *  0 <= rows < 2^31, dim 1..16384, eps > 0
 * Outputs overlap no input, except that r may be exactly the residual, in
 * place (dense rows), and each other not at all. */
int ssm_layer_norm_fwd(const void *x, int64_t x_stride, const void *residual,
                       int64_t residual_stride, const float *weight, const float *bias, void *r,
                       void *y, int64_t rows, int64_t dim, float eps, int x_dtype,
                       int residual_dtype, int dtype, void *stream);

/* Bytes of device workspace for ssm_layer_norm_bwd: partial sums of the
 * gradients of weight and bias. */
int ssm_layer_norm_bwd_workspace_size(int64_t rows, int64_t dim, size_t *bytes);

/* Gradients of ssm_layer_norm_fwd from its inputs (r and its mean and variance
 * are formed again) for gradients dr of r and dy of y.  With h = (r - mean) s,
 * s = 1 / sqrt(var + eps), g = dy weight:
 *   D = dr + s (g - mean(g) - h mean(g h))     the gradient of x and the residual
 *   dweight = sum over rows of dy h,   dbias = sum over rows of dy
 * A caller that kept r alone gives it as x, without a residual.
 *  dr         nullable (zero), residual_dtype (rows, dim) dense
 *  dy         required, dtype (rows, dim) dense
 *  dx         required output, x_dtype (rows, dim) dense: D
 *  dresidual  nullable output, residual_dtype (rows, dim) dense: D; only with a
 *             residual
 *  dweight    nullable output, fp32 (dim); also where weight is NULL
 *  dbias      nullable output, fp32 (dim)
 *  workspace  >= ssm_layer_norm_bwd_workspace_size() bytes, 256-byte aligned;
 *             its contents on entry do not matter
 * Outputs overlap nothing. */
int ssm_layer_norm_bwd(const void *x, int64_t x_stride, const void *residual,
                       int64_t residual_stride, const float *weight, const void *dr,
                       const void *dy, void *dx, void *dresidual, float *dweight, float *dbias,
                       int64_t rows, int64_t dim, float eps, int x_dtype, int residual_dtype,
                       int dtype, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------- the gradients' norm and clipping --
 * Over all elements g of n tensors: norm = sqrt(sum g^2), and
 * g' = g * min(1, max_norm / norm).  Each tensor is `sizes[i]` dense elements
 * at grads[i], of type dtypes[i]; the four arrays of pointers, sizes and types
 * are HOST arrays, read before the call returns.  Squares are summed in 64
 * bits, so that neither large nor small elements are lost.
 *  n >= 0, sizes[i] >= 0 (grads[i] may be NULL where it is 0)
 *  workspace  >= ssm_grad_workspace_size() bytes, 256-byte aligned, in use
 *             until the enqueued work is done; its contents on entry do not
 *             matter */
int ssm_grad_workspace_size(size_t *bytes);

/* norm: required output, one fp32. */
int ssm_grad_norm(const void *const *grads, const int64_t *sizes, const int *dtypes, int64_t n,
                  float *norm, void *workspace, size_t workspace_bytes, void *stream);

/* Clipping.
 *  outs, out_dtypes  NULL both: in place.  Else the clipped gradients' places
 *            and types, which may differ from the gradients'; outs[i] is
 *            grads[i] itself (of the same type) or overlaps no gradient
 *  max_norm  >= 0, or infinity (no clipping)
 *  have_norm nonzero: `norm` is read instead of formed (a norm that was summed
 *            over several processes); the workspace is then not used and may
 *            be NULL
 *  norm      required, one fp32; written unless have_norm
 * Where the norm is not finite the gradients stay as they are (outs get
 * copies), and the caller finds it in `norm`.  The factor is formed in 64 bits
 * and rounded to fp32.  No two gradients and no two outputs may overlap (a
 * tensor that is given twice would be clipped twice). */
int ssm_grad_clip(const void *const *grads, const int64_t *sizes, const int *dtypes,
                  void *const *outs, const int *out_dtypes, int64_t n, float max_norm,
                  int have_norm, float *norm, void *workspace, size_t workspace_bytes,
                  void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SSM_MODEL_H */
