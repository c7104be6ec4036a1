// ssm_model_api.cpp -- the C ABI of include/ssm_model.h: argument checks,
// workspaces and the tables of tensors.  Every check runs before the first HIP
// call.
#include "ssm_model.h"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <vector>

#include "ssm_internal.h"
#include "ssm_model_internal.h"

namespace {

int fail(int status, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return ssm::set_error(status, buf);
}

int ok() { return ssm::set_error(SSM_OK, ""); }

int done(int err) {
  if (err == 0) return ok();
  return fail(SSM_ERR_HIP, "kernel launch failed: %s", ssm::hip_error_string(err));
}

bool aligned(const void *p, size_t k) { return reinterpret_cast<uintptr_t>(p) % k == 0; }

int64_t size_of(int dtype) { return dtype == SSM_DTYPE_BF16 ? 2 : 4; }

bool is_dtype(int dtype) { return dtype == SSM_DTYPE_F32 || dtype == SSM_DTYPE_BF16; }

// An array of the call: n bytes from p (nothing if p is null).
struct Span {
  const void *p;
  int64_t n;
  const char *name;
};

bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  const char *x = static_cast<const char *>(a.p), *y = static_cast<const char *>(b.p);
  return x < y + b.n && y < x + a.n;
}

// Outputs overlap neither inputs nor each other.
template <int kI, int kO>
int check_overlaps(const Span (&ins)[kI], const Span (&outs)[kO]) {
  for (int o = 0; o < kO; ++o) {
    for (int i = 0; i < kI; ++i)
      if (overlap(outs[o], ins[i]))
        return fail(SSM_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, ins[i].name);
    for (int k = 0; k < o; ++k)
      if (overlap(outs[o], outs[k]))
        return fail(SSM_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, outs[k].name);
  }
  return SSM_OK;
}

int check_workspace(const void *workspace, size_t have, int64_t need) {
  if (need == 0) return SSM_OK;
  if (!workspace || have < static_cast<size_t>(need))
    return fail(SSM_ERR_WORKSPACE, "workspace of %lld bytes needed (got %zu bytes at %p)",
                (long long)need, have, workspace);
  if (!aligned(workspace, 256))
    return fail(SSM_ERR_INVALID_ARG, "workspace %p not 256-byte aligned", workspace);
  return SSM_OK;
}

constexpr int64_t kMaxStride = int64_t(1) << 22;

// Rows of dim elements, `stride` apart.
int check_rows(const char *name, const void *p, int64_t stride, int64_t dim, int dtype) {
  if (stride < dim)
    return fail(SSM_ERR_INVALID_ARG, "%s_stride=%lld is less than a row", name, (long long)stride);
  if (stride > kMaxStride)
    return fail(SSM_ERR_UNSUPPORTED, "%s_stride=%lld: this build supports up to %lld", name,
                (long long)stride, (long long)kMaxStride);
  if (!aligned(p, size_of(dtype)))
    return fail(SSM_ERR_INVALID_ARG, "%s=%p not aligned to its elements", name, p);
  return SSM_OK;
}

int64_t span_of(int64_t rows, int64_t stride, int64_t dim, int dtype) {
  return rows == 0 ? 0 : ((rows - 1) * stride + dim) * size_of(dtype);
}

// ------------------------------------------------------------- embedding --
constexpr int64_t kMaxTokens = (int64_t(1) << 28) - 1, kMaxVocab = (int64_t(1) << 30) - 1;

int check_embed_sizes(int64_t tokens, int64_t vocab, int64_t dim) {
  if (tokens < 0 || vocab <= 0 || dim <= 0)
    return fail(SSM_ERR_INVALID_ARG, "sizes out of range (tokens=%lld vocab=%lld dim=%lld)",
                (long long)tokens, (long long)vocab, (long long)dim);
  if (tokens > kMaxTokens || vocab > kMaxVocab || dim > ssm::kEmbedMaxDim)
    return fail(SSM_ERR_UNSUPPORTED, "tokens=%lld vocab=%lld dim=%lld: this build supports %lld, "
                "%lld and %d", (long long)tokens, (long long)vocab, (long long)dim,
                (long long)kMaxTokens, (long long)kMaxVocab, ssm::kEmbedMaxDim);
  if (tokens * dim > kMaxTokens * 1024)
    return fail(SSM_ERR_UNSUPPORTED, "tokens=%lld dim=%lld: this build supports %lld elements",
                (long long)tokens, (long long)dim, (long long)(kMaxTokens * 1024));
  return SSM_OK;
}

int check_embed(const void *ids, int64_t tokens, int64_t vocab, int64_t dim, float scale,
                int index_type, int dtype, int weight_dtype) {
  const int st = check_embed_sizes(tokens, vocab, dim);
  if (st != SSM_OK) return st;
  if (index_type != SSM_INDEX_I32 && index_type != SSM_INDEX_I64)
    return fail(SSM_ERR_INVALID_ARG, "unknown index type %d", index_type);
  if (!is_dtype(dtype) || !is_dtype(weight_dtype))
    return fail(SSM_ERR_INVALID_ARG, "unknown dtype (%d, %d)", dtype, weight_dtype);
  if (!std::isfinite(scale)) return fail(SSM_ERR_INVALID_ARG, "scale=%g is not finite", scale);
  if (tokens > 0 && !ids) return fail(SSM_ERR_INVALID_ARG, "ids is NULL");
  if (!aligned(ids, index_type == SSM_INDEX_I64 ? 8 : 4))
    return fail(SSM_ERR_INVALID_ARG, "ids=%p not aligned", ids);
  return SSM_OK;
}

// ------------------------------------------------------------ layer norm --
int check_norm_sizes(int64_t rows, int64_t dim) {
  if (rows < 0 || dim <= 0)
    return fail(SSM_ERR_INVALID_ARG, "sizes out of range (rows=%lld dim=%lld)", (long long)rows,
                (long long)dim);
  if (rows >= int64_t(1) << 31 || dim > ssm::kLayerNormMaxDim)
    return fail(SSM_ERR_UNSUPPORTED, "rows=%lld dim=%lld: this build supports under 2^31 and up to "
                "%d", (long long)rows, (long long)dim, ssm::kLayerNormMaxDim);
  return SSM_OK;
}

struct NormCall {
  const void *x, *residual;
  int64_t x_stride, r_stride;
  const float *weight, *bias;
  int64_t rows, dim;
  float eps;
  int xt, rt, yt;
};

int check_norm(const NormCall &c) {
  int st = check_norm_sizes(c.rows, c.dim);
  if (st != SSM_OK) return st;
  if (!is_dtype(c.xt) || !is_dtype(c.rt) || !is_dtype(c.yt))
    return fail(SSM_ERR_INVALID_ARG, "unknown dtype (%d, %d, %d)", c.xt, c.rt, c.yt);
  if (c.xt == SSM_DTYPE_BF16 ? c.yt != SSM_DTYPE_BF16 : c.rt != SSM_DTYPE_F32)
    return fail(SSM_ERR_INVALID_ARG, "x_dtype=%d residual_dtype=%d dtype=%d do not go together",
                c.xt, c.rt, c.yt);
  if (!c.residual && c.rt != c.xt && c.rows > 0)
    return fail(SSM_ERR_INVALID_ARG, "residual_dtype=%d without a residual: that of x (%d)", c.rt,
                c.xt);
  if (!(c.eps > 0.0f) || !std::isfinite(c.eps))
    return fail(SSM_ERR_INVALID_ARG, "eps=%g must be positive", c.eps);
  if (c.rows > 0 && !c.x) return fail(SSM_ERR_INVALID_ARG, "x is NULL");
  if ((st = check_rows("x", c.x, c.x_stride, c.dim, c.xt)) != SSM_OK) return st;
  if (c.residual && (st = check_rows("residual", c.residual, c.r_stride, c.dim, c.rt)) != SSM_OK)
    return st;
  if (!aligned(c.weight, 4) || !aligned(c.bias, 4))
    return fail(SSM_ERR_INVALID_ARG, "weight or bias not 4-byte aligned");
  return SSM_OK;
}

ssm::LayerNormTypes types_of(const NormCall &c) {
  if (c.xt == SSM_DTYPE_F32) return c.yt == SSM_DTYPE_F32 ? ssm::kLnF32 : ssm::kLnF32Bf16;
  return c.rt == SSM_DTYPE_F32 ? ssm::kLnBf16Wide : ssm::kLnBf16;
}

ssm::LayerNormArgs norm_args(const NormCall &c) {
  ssm::LayerNormArgs a{};
  a.x = c.x;
  a.residual = c.residual;
  a.x_stride = c.x_stride;
  a.r_stride = c.r_stride;
  a.weight = c.weight;
  a.bias = c.bias;
  a.rows = c.rows;
  a.dim = static_cast<int>(c.dim);
  a.eps = c.eps;
  return a;
}

int64_t norm_workspace(int64_t rows, int64_t dim) {
  return int64_t(ssm::layer_norm_bwd_parts(rows, static_cast<int>(dim))) * 2 * dim * 4;
}

// -------------------------------------------------------- gradients' norm --
constexpr int64_t kMaxGradSize = int64_t(1) << 40, kMaxGrads = int64_t(1) << 24;
constexpr int64_t kGradWorkspace = ssm::kGradGroups * 8;

struct Grads {
  const void *const *grads;
  const int64_t *sizes;
  const int *dtypes;
  void *const *outs;       // null: in place or none
  const int *out_dtypes;
  int64_t n;
};

int check_grads(const Grads &c) {
  if (c.n < 0) return fail(SSM_ERR_INVALID_ARG, "n=%lld", (long long)c.n);
  if (c.n > kMaxGrads)
    return fail(SSM_ERR_UNSUPPORTED, "n=%lld: this build supports up to %lld", (long long)c.n,
                (long long)kMaxGrads);
  if (c.n > 0 && (!c.grads || !c.sizes || !c.dtypes))
    return fail(SSM_ERR_INVALID_ARG, "grads, sizes or dtypes is NULL");
  if ((c.outs != nullptr) != (c.out_dtypes != nullptr) && c.n > 0)
    return fail(SSM_ERR_INVALID_ARG, "outs and out_dtypes go together");
  for (int64_t i = 0; i < c.n; ++i) {
    if (c.sizes[i] < 0)
      return fail(SSM_ERR_INVALID_ARG, "sizes[%lld]=%lld", (long long)i, (long long)c.sizes[i]);
    if (c.sizes[i] >= kMaxGradSize)
      return fail(SSM_ERR_UNSUPPORTED, "sizes[%lld]=%lld: too large", (long long)i,
                  (long long)c.sizes[i]);
    if (!is_dtype(c.dtypes[i]) || (c.outs && !is_dtype(c.out_dtypes[i])))
      return fail(SSM_ERR_INVALID_ARG, "unknown dtype of tensor %lld", (long long)i);
    if (c.sizes[i] == 0) continue;
    if (!c.grads[i] || (c.outs && !c.outs[i]))
      return fail(SSM_ERR_INVALID_ARG, "tensor %lld is NULL", (long long)i);
    if (!aligned(c.grads[i], size_of(c.dtypes[i])) ||
        (c.outs && !aligned(c.outs[i], size_of(c.out_dtypes[i]))))
      return fail(SSM_ERR_INVALID_ARG, "tensor %lld not aligned to its elements", (long long)i);
  }
  return SSM_OK;
}

// No two written arrays overlap, and none overlaps another's gradient; two
// gradients that are only read may be the same.
struct Range {
  uintptr_t from, to;
  int64_t i;
  bool written;
};

int check_grad_overlaps(const Grads &c, bool clip, const Span *more, int nmore) {
  if (!clip && nmore == 0) return SSM_OK;
  std::vector<Range> v;
  v.reserve(static_cast<size_t>(c.n) * 2 + nmore);
  auto add = [&](const void *p, int64_t bytes, int64_t i, bool written) {
    if (!p || bytes <= 0) return;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    v.push_back({at, at + static_cast<uintptr_t>(bytes), i, written});
  };
  for (int64_t i = 0; i < c.n; ++i) {
    const int64_t bytes = c.sizes[i] * size_of(c.dtypes[i]);
    const bool own = clip && (!c.outs || (c.outs[i] == c.grads[i] &&
                                          c.out_dtypes[i] == c.dtypes[i]));
    add(c.grads[i], bytes, i, own);
    if (clip && !own) add(c.outs[i], c.sizes[i] * size_of(c.out_dtypes[i]), i, true);
  }
  for (int k = 0; k < nmore; ++k) add(more[k].p, more[k].n, -1 - k, true);
  std::sort(v.begin(), v.end(), [](const Range &a, const Range &b) { return a.from < b.from; });
  // the furthest end so far, of written and of all ranges
  uintptr_t end_all = 0, end_written = 0;
  int64_t who_all = 0, who_written = 0;
  for (const Range &r : v) {
    const bool bad_read = r.from < end_written, bad_write = r.written && r.from < end_all;
    if (bad_read || bad_write) {
      const int64_t other = bad_read ? who_written : who_all;
      if (r.i < 0 || other < 0)
        return fail(SSM_ERR_INVALID_ARG, "norm or workspace overlaps a tensor or each other");
      return fail(SSM_ERR_INVALID_ARG, "tensors %lld and %lld overlap", (long long)other,
                  (long long)r.i);
    }
    if (r.to > end_all) end_all = r.to, who_all = r.i;
    if (r.written && r.to > end_written) end_written = r.to, who_written = r.i;
  }
  // two gradients that are clipped to two places may not be one either
  if (clip && c.outs) {
    end_all = 0;
    for (const Range &r : v) {
      if (r.i < 0) continue;
      const bool grad = reinterpret_cast<uintptr_t>(c.grads[r.i]) == r.from;
      if (!grad) continue;
      if (r.from < end_all)
        return fail(SSM_ERR_INVALID_ARG, "gradient %lld overlaps another", (long long)r.i);
      end_all = std::max(end_all, r.to);
    }
  }
  return SSM_OK;
}

int64_t chunks_of(int64_t size, int64_t chunk) { return (size + chunk - 1) / chunk; }

// The tensors of a call as entries of at most kGradPiece elements, in tables of
// equal numbers of entries.
struct Tables {
  std::vector<ssm::GradTable> t;
  std::vector<ssm::GradOuts> o;
  int groups = 1;  // workgroups, and sums, of a launch
  bool small;      // one table, of pieces

  // form_norm: the norm is formed, by one workgroup where it can
  Tables(const Grads &c, bool form_norm) {
    int64_t entries = 0, pieces = 0;
    for (int64_t i = 0; i < c.n; ++i) {
      entries += chunks_of(c.sizes[i], ssm::kGradPiece);
      pieces += chunks_of(c.sizes[i], 8);
    }
    small = form_norm && entries <= ssm::kGradTensors && pieces <= ssm::kGradSmall;
    const int64_t chunk = small ? 8 : ssm::kGradChunk;
    const int64_t tables = std::max<int64_t>(1, (entries + ssm::kGradTensors - 1) / ssm::kGradTensors);
    const int64_t each = (entries + tables - 1) / tables;
    t.resize(tables);
    o.resize(tables);
    int64_t k = 0;
    for (auto &table : t) table.n = 0, table.first[0] = 0;
    for (int64_t i = 0; i < c.n; ++i) {
      const int in = c.dtypes[i], out = c.outs ? c.out_dtypes[i] : in;
      const char *g = static_cast<const char *>(c.grads[i]);
      char *w = static_cast<char *>(c.outs ? c.outs[i] : const_cast<void *>(c.grads[i]));
      for (int64_t at = 0; at < c.sizes[i]; at += ssm::kGradPiece) {
        if (t[k].n == each) ++k;
        ssm::GradTable &table = t[k];
        const int64_t size = std::min(c.sizes[i] - at, ssm::kGradPiece);
        table.grad[table.n] = g + at * size_of(in);
        o[k].out[table.n] = w + at * size_of(out);
        table.size[table.n] = static_cast<uint32_t>(size) |
                              (in == SSM_DTYPE_BF16 ? ssm::kGradBf16 : 0u) |
                              (out == SSM_DTYPE_BF16 ? ssm::kGradOutBf16 : 0u);
        table.first[table.n + 1] = table.first[table.n] + static_cast<uint32_t>(chunks_of(size, chunk));
        ++table.n;
      }
    }
    uint32_t most = 1;
    for (const auto &table : t) most = std::max(most, table.first[table.n]);
    groups = static_cast<int>(std::min<uint32_t>(most, ssm::kGradGroups));
  }
};

int form_squares(const Tables &t, double *sums, void *stream) {
  for (size_t i = 0; i < t.t.size(); ++i) {
    const int err = ssm::launch_grad_squares(t.t[i], sums, t.groups, i == 0, stream);
    if (err != 0) return err;
  }
  return 0;
}

}  // namespace

extern "C" {

int ssm_embed_fwd(const void *ids, const void *weight, int64_t weight_stride, void *out,
                  int64_t tokens, int64_t vocab, int64_t dim, float scale, int index_type,
                  int weight_dtype, int dtype, void *stream) {
  int st = check_embed(ids, tokens, vocab, dim, scale, index_type, dtype, weight_dtype);
  if (st != SSM_OK) return st;
  if ((st = check_rows("weight", weight, weight_stride, dim, weight_dtype)) != SSM_OK) return st;
  if (tokens == 0) return ok();
  if (!weight || !out) return fail(SSM_ERR_INVALID_ARG, "weight or out is NULL");
  if (!aligned(out, size_of(dtype))) return fail(SSM_ERR_INVALID_ARG, "out=%p not aligned", out);
  const Span ins[] = {{ids, tokens * (index_type == SSM_INDEX_I64 ? 8 : 4), "ids"},
                      {weight, span_of(vocab, weight_stride, dim, weight_dtype), "weight"}};
  const Span outs[] = {{out, tokens * dim * size_of(dtype), "out"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;
  ssm::EmbedArgs a{};
  a.ids = ids;
  a.wide_ids = index_type == SSM_INDEX_I64;
  a.tokens = tokens;
  a.vocab = vocab;
  a.dim = static_cast<int>(dim);
  a.scale = scale;
  a.weight = weight;
  a.w_stride = weight_stride;
  a.out = out;
  return done(ssm::launch_embed_fwd(a, weight_dtype == SSM_DTYPE_BF16, dtype == SSM_DTYPE_BF16,
                                    stream));
}

int ssm_embed_bwd_workspace_size(int64_t tokens, int64_t vocab, int64_t dim, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "bytes is NULL");
  const int st = check_embed_sizes(tokens, vocab, dim);
  if (st != SSM_OK) return st;
  *bytes = static_cast<size_t>(ssm::embed_bwd_workspace(tokens, dim));
  return ok();
}

int ssm_embed_bwd(const void *ids, const void *dy, int64_t dy_stride, void *dweight,
                  int64_t tokens, int64_t vocab, int64_t dim, float scale, unsigned flags,
                  int index_type, int dtype, int weight_dtype, void *workspace,
                  size_t workspace_bytes, void *stream) {
  int st = check_embed(ids, tokens, vocab, dim, scale, index_type, dtype, weight_dtype);
  if (st != SSM_OK) return st;
  if (flags & ~SSM_FLAG_ACCUMULATE) return fail(SSM_ERR_INVALID_ARG, "unknown flags %#x", flags);
  if ((st = check_rows("dy", dy, dy_stride, dim, dtype)) != SSM_OK) return st;
  if ((tokens > 0 && !dy) || !dweight) return fail(SSM_ERR_INVALID_ARG, "dy or dweight is NULL");
  if (!aligned(dweight, size_of(weight_dtype)))
    return fail(SSM_ERR_INVALID_ARG, "dweight=%p not aligned", dweight);
  const int64_t need = ssm::embed_bwd_workspace(tokens, dim);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != SSM_OK) return st;
  const Span ins[] = {{ids, tokens * (index_type == SSM_INDEX_I64 ? 8 : 4), "ids"},
                      {dy, span_of(tokens, dy_stride, dim, dtype), "dy"}};
  const Span outs[] = {{dweight, vocab * dim * size_of(weight_dtype), "dweight"},
                       {workspace, need, "workspace"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;
  ssm::EmbedArgs a{};
  a.ids = ids;
  a.wide_ids = index_type == SSM_INDEX_I64;
  a.tokens = tokens;
  a.vocab = vocab;
  a.dim = static_cast<int>(dim);
  a.scale = scale;
  a.dy = dy;
  a.dy_stride = dy_stride;
  a.dweight = dweight;
  a.accumulate = (flags & SSM_FLAG_ACCUMULATE) != 0;
  a.workspace = workspace;
  return done(ssm::launch_embed_bwd(a, weight_dtype == SSM_DTYPE_BF16, dtype == SSM_DTYPE_BF16,
                                    stream));
}

int ssm_layer_norm_fwd(const void *x, int64_t x_stride, const void *residual,
                       int64_t residual_stride, const float *weight, const float *bias, void *r,
                       void *y, int64_t rows, int64_t dim, float eps, int x_dtype,
                       int residual_dtype, int dtype, void *stream) {
  const NormCall c{x, residual, x_stride, residual_stride, weight, bias, rows, dim, eps, x_dtype,
                   residual_dtype, dtype};
  int st = check_norm(c);
  if (st != SSM_OK) return st;
  if (rows == 0) return ok();
  if (!y) return fail(SSM_ERR_INVALID_ARG, "y is NULL");
  if (r && !residual) return fail(SSM_ERR_INVALID_ARG, "r without a residual");
  if (!aligned(r, size_of(residual_dtype)) || !aligned(y, size_of(dtype)))
    return fail(SSM_ERR_INVALID_ARG, "output not aligned (r=%p y=%p)", r, y);
  const bool in_place = r && r == residual && residual_stride == dim;
  const Span ins[] = {{x, span_of(rows, x_stride, dim, x_dtype), "x"},
                      {in_place ? nullptr : residual,
                       span_of(rows, residual_stride, dim, residual_dtype), "residual"},
                      {weight, dim * 4, "weight"}, {bias, dim * 4, "bias"}};
  const Span outs[] = {{r, rows * dim * size_of(residual_dtype), "r"},
                       {y, rows * dim * size_of(dtype), "y"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;
  ssm::LayerNormArgs a = norm_args(c);
  a.r = r;
  a.y = y;
  return done(ssm::launch_layer_norm_fwd(a, types_of(c), stream));
}

int ssm_layer_norm_bwd_workspace_size(int64_t rows, int64_t dim, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "bytes is NULL");
  const int st = check_norm_sizes(rows, dim);
  if (st != SSM_OK) return st;
  *bytes = static_cast<size_t>(norm_workspace(rows, dim));
  return ok();
}

int ssm_layer_norm_bwd(const void *x, int64_t x_stride, const void *residual,
                       int64_t residual_stride, const float *weight, const void *dr,
                       const void *dy, void *dx, void *dresidual, float *dweight, float *dbias,
                       int64_t rows, int64_t dim, float eps, int x_dtype, int residual_dtype,
                       int dtype, void *workspace, size_t workspace_bytes, void *stream) {
  const NormCall c{x, residual, x_stride, residual_stride, weight, nullptr, rows, dim, eps,
                   x_dtype, residual_dtype, dtype};
  int st = check_norm(c);
  if (st != SSM_OK) return st;
  if (dresidual && !residual && rows > 0)
    return fail(SSM_ERR_INVALID_ARG, "dresidual without a residual");
  if (rows > 0 && (!dy || !dx)) return fail(SSM_ERR_INVALID_ARG, "dy or dx is NULL");
  if (!aligned(dr, size_of(residual_dtype)) || !aligned(dresidual, size_of(residual_dtype)) ||
      !aligned(dy, size_of(dtype)) || !aligned(dx, size_of(x_dtype)))
    return fail(SSM_ERR_INVALID_ARG, "activation pointer not aligned");
  if (!aligned(dweight, 4) || !aligned(dbias, 4))
    return fail(SSM_ERR_INVALID_ARG, "weight gradients not 4-byte aligned");
  const int64_t need = norm_workspace(rows, dim);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != SSM_OK) return st;
  const int64_t all = rows * dim;
  const Span ins[] = {{x, span_of(rows, x_stride, dim, x_dtype), "x"},
                      {residual, span_of(rows, residual_stride, dim, residual_dtype), "residual"},
                      {weight, dim * 4, "weight"}, {dr, all * size_of(residual_dtype), "dr"},
                      {dy, all * size_of(dtype), "dy"}};
  const Span outs[] = {{dx, all * size_of(x_dtype), "dx"},
                       {dresidual, all * size_of(residual_dtype), "dresidual"},
                       {dweight, dim * 4, "dweight"}, {dbias, dim * 4, "dbias"},
                       {workspace, need, "workspace"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;
  ssm::LayerNormArgs a = norm_args(c);
  a.dr = dr;
  a.dy = dy;
  a.dx = dx;
  a.dresidual = dresidual;
  a.dweight = dweight;
  a.dbias = dbias;
  a.parts = static_cast<float *>(workspace);
  return done(ssm::launch_layer_norm_bwd(a, types_of(c), stream));
}

int ssm_grad_workspace_size(size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = kGradWorkspace;
  return ok();
}

int ssm_grad_norm(const void *const *grads, const int64_t *sizes, const int *dtypes, int64_t n,
                  float *norm, void *workspace, size_t workspace_bytes, void *stream) try {
  const Grads c{grads, sizes, dtypes, nullptr, nullptr, n};
  int st = check_grads(c);
  if (st != SSM_OK) return st;
  if (!norm || !aligned(norm, 4)) return fail(SSM_ERR_INVALID_ARG, "norm=%p", (void *)norm);
  if ((st = check_workspace(workspace, workspace_bytes, kGradWorkspace)) != SSM_OK) return st;
  const Span more[] = {{norm, 4, "norm"}, {workspace, kGradWorkspace, "workspace"}};
  if ((st = check_grad_overlaps(c, false, more, 2)) != SSM_OK) return st;
  double *sums = static_cast<double *>(workspace);
  const Tables t(c, true);
  if (t.small)
    return done(ssm::launch_grad_small(t.t[0], t.o[0], false, false, 0.0f, norm, stream));
  const int err = form_squares(t, sums, stream);
  return done(err != 0 ? err : ssm::launch_grad_norm(sums, t.groups, norm, stream));
} catch (const std::bad_alloc &) {
  return fail(SSM_ERR_INVALID_ARG, "out of host memory");
}

int ssm_grad_clip(const void *const *grads, const int64_t *sizes, const int *dtypes,
                  void *const *outs, const int *out_dtypes, int64_t n, float max_norm,
                  int have_norm, float *norm, void *workspace, size_t workspace_bytes,
                  void *stream) try {
  const Grads c{grads, sizes, dtypes, outs, out_dtypes, n};
  int st = check_grads(c);
  if (st != SSM_OK) return st;
  if (!(max_norm >= 0.0f)) return fail(SSM_ERR_INVALID_ARG, "max_norm=%g", max_norm);
  if (!norm || !aligned(norm, 4)) return fail(SSM_ERR_INVALID_ARG, "norm=%p", (void *)norm);
  if (!have_norm &&
      (st = check_workspace(workspace, workspace_bytes, kGradWorkspace)) != SSM_OK)
    return st;
  const Span more[] = {{norm, 4, "norm"},
                       {have_norm ? nullptr : workspace, kGradWorkspace, "workspace"}};
  if ((st = check_grad_overlaps(c, true, more, 2)) != SSM_OK) return st;
  double *sums = have_norm ? nullptr : static_cast<double *>(workspace);
  const Tables t(c, !have_norm);
  if (t.small)
    return done(ssm::launch_grad_small(t.t[0], t.o[0], true, outs == nullptr, max_norm, norm, stream));
  int err = have_norm ? 0 : form_squares(t, sums, stream);
  // the tables from the last one, too, for the last-level cache
  for (size_t i = t.t.size(); i-- > 0 && err == 0;)
    err = ssm::launch_grad_scale(t.t[i], t.o[i], outs == nullptr, sums, t.groups, max_norm, norm,
                                 i == 0 && !have_norm, stream);
  return done(err);
} catch (const std::bad_alloc &) {
  return fail(SSM_ERR_INVALID_ARG, "out of host memory");
}

}  // extern "C"
