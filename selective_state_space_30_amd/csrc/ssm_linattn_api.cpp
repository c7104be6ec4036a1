// ssm_linattn_api.cpp -- the C ABI of include/ssm_linattn.h: argument checks,
// how the sequences are cut, workspaces, and the order of the kernels.  Every
// check runs before the first HIP call.
#include "ssm_linattn.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ssm_block_norm.h"
#include "ssm_internal.h"
#include "ssm_linattn_internal.h"

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

int hip_failed(int err) {
  return fail(SSM_ERR_HIP, "kernel launch failed: %s", ssm::hip_error_string(err));
}

bool aligned(const void *p, size_t k) { return reinterpret_cast<uintptr_t>(p) % k == 0; }

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

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

int check_workspace(const void *workspace, size_t have, size_t need) {
  if (need == 0) return SSM_OK;
  if (!workspace || have < need)
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu bytes at %p)", need,
                have, workspace);
  if (!aligned(workspace, 256))
    return fail(SSM_ERR_INVALID_ARG, "workspace %p not 256-byte aligned", workspace);
  return SSM_OK;
}

// Row strides: a chunk of rows is addressed by 32-bit byte offsets.
constexpr int64_t kMaxStride = int64_t(1) << 22;

// Workgroups of 256 threads a launch may have (2^32 threads).
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;

// ------------------------------------------------------ linear attention --
struct Sizes {
  int64_t tokens, nseq, heads, qk_heads, dk, dv;
  int dtype;
  bool packed;
  bool bf16() const { return dtype == SSM_DTYPE_BF16; }
  int64_t es() const { return bf16() ? 2 : 4; }
};

int check_sizes(const Sizes &z) {
  if (z.dtype != SSM_DTYPE_F32 && z.dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_INVALID_ARG, "unknown dtype %d", z.dtype);
  if (z.tokens < 0 || z.nseq <= 0 || z.heads <= 0 || z.qk_heads <= 0 || z.dk <= 0 || z.dv <= 0)
    return fail(SSM_ERR_INVALID_ARG,
                "sizes out of range (tokens=%lld nseq=%lld heads=%lld qk_heads=%lld qk_dim=%lld "
                "v_dim=%lld)",
                (long long)z.tokens, (long long)z.nseq, (long long)z.heads,
                (long long)z.qk_heads, (long long)z.dk, (long long)z.dv);
  if (z.heads % z.qk_heads != 0)
    return fail(SSM_ERR_INVALID_ARG, "heads=%lld is no multiple of qk_heads=%lld",
                (long long)z.heads, (long long)z.qk_heads);
  if (z.dk > ssm::kLinMaxDim || z.dv > ssm::kLinMaxDim)
    return fail(SSM_ERR_UNSUPPORTED, "qk_dim=%lld v_dim=%lld: this build supports 1..%d",
                (long long)z.dk, (long long)z.dv, ssm::kLinMaxDim);
  if (z.tokens >= (int64_t(1) << 31) || z.nseq >= (int64_t(1) << 31) || z.heads > 65536)
    return fail(SSM_ERR_UNSUPPORTED, "tokens=%lld nseq=%lld heads=%lld: too large",
                (long long)z.tokens, (long long)z.nseq, (long long)z.heads);
  if (!z.packed && z.tokens % z.nseq != 0)
    return fail(SSM_ERR_INVALID_ARG, "tokens=%lld is no multiple of nseq=%lld without cu_seqlens",
                (long long)z.tokens, (long long)z.nseq);
  return SSM_OK;
}

// Segments.  A sequence's chunks follow one another, so that one segment a
// sequence leaves as many workgroups as there are heads (or pairs of them)
// and column slices.  Where they fill the GPU's places for workgroups less
// than half, the sequences are cut into as many segments of at least
// kMinSegment tokens as fill them once, for the price of a pass over k and v
// (and q and do) that forms the states between them.  A CU holds two
// workgroups, or one of heads over 128 wide.  Measured with 256, 512 and 1024
// places: prompts of 2 x 4096 tokens, 80 heads of 64 on states of 128, 170,
// 150 and 172 us; one of 65536 tokens, 8 heads of 128, 241, 224 and 258 us;
// with segments of at least 128, 256 and 512 tokens: 7 short fp32 prompts
// 103, 176 and 333 us, a training step of 2 x 2048 tokens 181, 173 and 186 us.
// The gradient of the decay is summed over one segment in 64 bits from an
// inner product at its end, so with it segments have at most
// kMaxGradSegment tokens.
constexpr int64_t kPlaces = 512, kMinSegment = 128, kMaxGradSegment = 1024;

// workgroups that `out` output columns take
int64_t slices_of(int64_t out) {
  const int64_t w = ssm::linattn_slice(static_cast<int>(out));
  return (out + w - 1) / w;
}

// value heads that a workgroup takes
int64_t heads_per_group(const Sizes &z) {
  return ssm::linattn_pairs_heads(static_cast<int>(z.heads / z.qk_heads), static_cast<int>(z.dv))
             ? 2 : 1;
}

// workgroups that a sequence's chunk pass has
int64_t groups_of(const Sizes &z, bool backward) {
  const int64_t one = z.heads / heads_per_group(z) * slices_of(z.dv);
  return backward ? one + 2 * z.heads * slices_of(z.dk) : one;
}

ssm::LinPlan make_plan(const Sizes &z, bool backward, bool decay_grad) {
  const int64_t chunk = ssm::linattn_chunk(z.bf16());
  const int64_t longest = z.packed ? z.tokens : z.tokens / z.nseq;
  const int64_t groups = groups_of(z, backward);
  const int64_t places = z.dk > 128 || (backward && z.dv > 128) ? kPlaces / 2 : kPlaces;
  int64_t seg = up(longest > 0 ? longest : 1, chunk);
  if (z.packed) {
    // sequences may differ in length: their tokens count, not their number
    const int64_t cut = up((z.tokens * groups + places - 1) / places, chunk);
    if (cut < seg) seg = cut > kMinSegment ? cut : kMinSegment;
    if (seg > longest) seg = up(longest > 0 ? longest : 1, chunk);
  } else {
    int64_t segs = places / (z.nseq * groups);
    if (segs > longest / kMinSegment) segs = longest / kMinSegment;
    if (segs > 1) seg = up((longest + segs - 1) / segs, chunk);
  }
  if (decay_grad && seg > kMaxGradSegment) seg = kMaxGradSegment;
  ssm::LinPlan p{};
  p.tokens = z.tokens;
  p.seqlen = z.packed ? 0 : z.tokens / z.nseq;
  p.seg_len = seg;
  p.segs = z.packed ? 0 : p.seqlen > seg ? (p.seqlen + seg - 1) / seg : 1;
  p.slots = z.packed ? z.tokens / seg + z.nseq : z.nseq * p.segs;
  p.nseq = static_cast<int>(z.nseq);
  p.heads = static_cast<int>(z.heads);
  return p;
}

bool many_segments(const Sizes &z, const ssm::LinPlan &p) {
  return z.packed ? p.seg_len < z.tokens : p.segs > 1;
}

// The plan of the sums over pairs, whose workgroups take a chunk each:
// segments of one chunk.  Their number grows with the tokens, not with the
// length that the segments happen to have.
ssm::LinPlan pairs_plan(const Sizes &z, ssm::LinPlan p) {
  const int64_t chunk = ssm::linattn_chunk(z.bf16());
  p.seg_len = chunk;
  p.segs = z.packed ? 0 : p.seqlen > chunk ? (p.seqlen + chunk - 1) / chunk : 1;
  p.slots = z.packed ? z.tokens / chunk + z.nseq : z.nseq * p.segs;
  return p;
}

// Whether every launch of the call stays within 2^32 threads.  backward: 0
// no, 1 yes, 2 with dg.
int check_plan(const Sizes &z, const ssm::LinPlan &p, int backward) {
  if (z.heads * z.dk > kMaxStride || z.heads * z.dv > kMaxStride)
    return fail(SSM_ERR_UNSUPPORTED, "heads=%lld: rows too long", (long long)z.heads);
  // the chain; and the widest of the others: the output pass, or the gradients'
  // three and with dg the pairs', all of at most 512 threads
  int64_t groups = p.slots * z.heads * slices_of(z.dv);
  if (backward) groups += 2 * p.slots * z.heads * slices_of(z.dk);
  if (backward == 2) groups += pairs_plan(z, p).slots * z.heads / heads_per_group(z);
  if (z.nseq * z.heads > kMaxGroups || 2 * groups > kMaxGroups)
    return fail(SSM_ERR_UNSUPPORTED, "tokens=%lld heads=%lld nseq=%lld: too many workgroups",
                (long long)z.tokens, (long long)z.heads, (long long)z.nseq);
  return SSM_OK;
}

struct FwdLayout {
  int64_t states, decay, total;
};

FwdLayout fwd_layout(const Sizes &z, const ssm::LinPlan &p) {
  FwdLayout l{};
  if (!many_segments(z, p)) return l;
  const int64_t cells = p.slots * z.heads;
  l.states = 0;
  l.decay = up(cells * z.dk * z.dv * 4, 256);
  l.total = l.decay + up(cells * 4, 256);
  return l;
}

struct BwdLayout {
  int64_t states, adjoints, decay, adecay, last, dq, dk, pairs, xdots, ydots, dg, total;
};

// want_dg: 0 no, 1 a token, 2 a head
BwdLayout bwd_layout(const Sizes &z, const ssm::LinPlan &p, int want_dg) {
  BwdLayout l{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  const int64_t size = z.dk * z.dv * 4, cells = p.slots * z.heads;
  if (many_segments(z, p)) {
    l.states = take(cells * size);
    l.adjoints = take(cells * size);
    l.decay = take(cells * 4);
    l.adecay = take(cells * 4);
  }
  if (z.qk_heads != z.heads) {
    l.dq = take(z.tokens * z.heads * z.dk * 4);
    l.dk = take(z.tokens * z.heads * z.dk * 4);
  }
  if (want_dg) {
    const int64_t one = z.tokens * z.heads * 4;
    l.last = take(z.nseq * z.heads * size);
    l.pairs = take(one);
    l.xdots = take(one * slices_of(z.dk));
    l.ydots = take(one * slices_of(z.dk));
    if (want_dg == 2) l.dg = take(one);
  }
  l.total = at;
  return l;
}

int check_stride(const char *name, int64_t stride, int64_t row) {
  if (stride < row)
    return fail(SSM_ERR_INVALID_ARG, "%s_stride=%lld: rows have %lld elements", name,
                (long long)stride, (long long)row);
  if (stride > kMaxStride)
    return fail(SSM_ERR_UNSUPPORTED, "%s_stride=%lld: this build supports up to %lld", name,
                (long long)stride, (long long)kMaxStride);
  return SSM_OK;
}

int64_t span_bytes(int64_t rows, int64_t stride, int64_t row, int64_t es) {
  return rows > 0 ? ((rows - 1) * stride + row) * es : 0;
}

struct Call {
  Sizes z;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *g, *h0;
  const int32_t *cu;
  unsigned flags;
  float scale;
};

int64_t g_bytes(const Call &c) {
  return (c.flags & SSM_FLAG_HEAD_DECAY ? 1 : c.z.tokens) * c.z.heads * 4;
}

int g_kind(const Call &c) {
  return !c.g ? ssm::kLinDecayNone
              : c.flags & SSM_FLAG_HEAD_DECAY ? ssm::kLinDecayHead : ssm::kLinDecayToken;
}

// The checks that the calls share; `flags`: those that this one takes.
int check_call(const Call &c, unsigned flags) {
  int st = check_sizes(c.z);
  if (st != SSM_OK) return st;
  if (c.flags & ~flags)
    return fail(SSM_ERR_INVALID_ARG, "unknown flag bits 0x%x", c.flags);
  if (c.z.tokens > 0 && (!c.q || !c.k || !c.v))
    return fail(SSM_ERR_INVALID_ARG, "required pointer is NULL (q=%p k=%p v=%p)", c.q, c.k, c.v);
  if (!std::isfinite(c.scale)) return fail(SSM_ERR_INVALID_ARG, "scale is not finite");
  if ((st = check_stride("q", c.q_stride, c.z.qk_heads * c.z.dk)) != SSM_OK) return st;
  if ((st = check_stride("k", c.k_stride, c.z.qk_heads * c.z.dk)) != SSM_OK) return st;
  if ((st = check_stride("v", c.v_stride, c.z.heads * c.z.dv)) != SSM_OK) return st;
  const void *acts[] = {c.q, c.k, c.v};
  for (const void *p : acts)
    if (!aligned(p, c.z.es()))
      return fail(SSM_ERR_INVALID_ARG, "activation pointer %p not %lld-byte aligned", p,
                  (long long)c.z.es());
  const void *words[] = {c.g, c.h0, c.cu};
  for (const void *p : words)
    if (!aligned(p, 4)) return fail(SSM_ERR_INVALID_ARG, "pointer %p not 4-byte aligned", p);
  return SSM_OK;
}

// Whether the call sets the rows outside its sequences to 0 (only packed
// ones leave any).
bool zero_outside(const Call &c) {
  return (c.flags & SSM_FLAG_ZERO_OUTSIDE) && c.cu && c.z.tokens > 0;
}

bool rows16(const void *p, int64_t stride, int64_t d, int64_t es) {
  return aligned(p, 16) && stride * es % 16 == 0 && d * es % 16 == 0;
}

ssm::LinSide side(const void *p, int64_t stride, int64_t d, int64_t div) {
  return ssm::LinSide{p, stride, static_cast<int>(d), static_cast<int>(div)};
}

}  // namespace

extern "C" {

int ssm_linattn_plan(int64_t tokens, int64_t nseq, int packed, int64_t heads, int64_t qk_heads,
                     int64_t qk_dim, int64_t v_dim, int dtype, int backward, int64_t *plan_out) {
  if (!plan_out) return fail(SSM_ERR_INVALID_ARG, "plan_out is NULL");
  if (backward < 0 || backward > 2)
    return fail(SSM_ERR_INVALID_ARG, "backward=%d: 0..2", backward);
  const Sizes z{tokens, nseq, heads, qk_heads, qk_dim, v_dim, dtype, packed != 0};
  int st = check_sizes(z);
  if (st != SSM_OK) return st;
  const ssm::LinPlan p = make_plan(z, backward != 0, backward == 2);
  if ((st = check_plan(z, p, backward)) != SSM_OK) return st;
  plan_out[0] = p.seg_len;
  plan_out[1] = p.slots;
  plan_out[2] = ssm::linattn_chunk(z.bf16());
  plan_out[3] = many_segments(z, p) ? 1 : 0;
  return ok();
}

int ssm_linattn_workspace_size(int64_t tokens, int64_t nseq, int packed, int64_t heads,
                               int64_t qk_heads, int64_t qk_dim, int64_t v_dim, int dtype,
                               size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "bytes is NULL");
  const Sizes z{tokens, nseq, heads, qk_heads, qk_dim, v_dim, dtype, packed != 0};
  int st = check_sizes(z);
  if (st != SSM_OK) return st;
  const ssm::LinPlan p = make_plan(z, false, false);
  if ((st = check_plan(z, p, 0)) != SSM_OK) return st;
  *bytes = static_cast<size_t>(fwd_layout(z, p).total);
  return ok();
}

int ssm_linattn_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const float *g, unsigned flags, float scale,
                    const float *h0, const int32_t *cu_seqlens, void *o, float *h_final,
                    int64_t tokens, int64_t nseq, int64_t heads, int64_t qk_heads, int64_t qk_dim,
                    int64_t v_dim, int dtype, void *workspace, size_t workspace_bytes,
                    void *stream) {
  const Call c{{tokens, nseq, heads, qk_heads, qk_dim, v_dim, dtype, cu_seqlens != nullptr},
               q, k, v, q_stride, k_stride, v_stride, g, h0, cu_seqlens, flags, scale};
  int st = check_call(c, SSM_FLAG_HEAD_DECAY | SSM_FLAG_ZERO_OUTSIDE);
  if (st != SSM_OK) return st;
  const Sizes &z = c.z;
  const int64_t es = z.es();
  if (tokens > 0 && !o) return fail(SSM_ERR_INVALID_ARG, "o is NULL");
  if (!aligned(o, es) || !aligned(h_final, 4))
    return fail(SSM_ERR_INVALID_ARG, "output not aligned (o=%p h_final=%p)", o, (void *)h_final);
  ssm::LinPlan plan = make_plan(z, false, false);
  if ((st = check_plan(z, plan, 0)) != SSM_OK) return st;
  const FwdLayout l = fwd_layout(z, plan);
  if ((st = check_workspace(workspace, workspace_bytes, static_cast<size_t>(l.total))) != SSM_OK)
    return st;
  const int64_t states = nseq * heads * qk_dim * v_dim * 4;
  const Span ins[] = {{q, span_bytes(tokens, q_stride, qk_heads * qk_dim, es), "q"},
                      {k, span_bytes(tokens, k_stride, qk_heads * qk_dim, es), "k"},
                      {v, span_bytes(tokens, v_stride, heads * v_dim, es), "v"},
                      {g, g_bytes(c), "g"},
                      {h0, states, "h0"},
                      {cu_seqlens, (nseq + 1) * 4, "cu_seqlens"}};
  const Span outs[] = {{o, tokens * heads * v_dim * es, "o"},
                       {h_final, states, "h_final"},
                       {workspace, l.total, "workspace"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;

  plan.cu = cu_seqlens;
  plan.vec = rows16(q, q_stride, qk_dim, es) && rows16(k, k_stride, qk_dim, es) &&
             rows16(v, v_stride, v_dim, es) && aligned(o, 16);
  const int64_t div = heads / qk_heads;
  ssm::LinCore a{};
  a.plan = plan;
  a.q = side(q, q_stride, qk_dim, div);
  a.k = side(k, k_stride, qk_dim, div);
  a.v = side(v, v_stride, v_dim, 1);
  a.g = g;
  a.g_kind = g_kind(c);
  a.inter = a.inside = scale;
  a.into = 1.0f;
  a.in_seqs = h0;
  a.sa = static_cast<int>(v_dim);
  a.sb = 1;
  int err;
  if (l.total) {
    char *w = static_cast<char *>(workspace);
    a.out_slots = reinterpret_cast<float *>(w + l.states);
    a.out_decay = reinterpret_cast<float *>(w + l.decay);
    err = z.bf16() ? ssm::launch_linattn_states_bf16(a, nullptr, stream)
                   : ssm::launch_linattn_states_f32(a, nullptr, stream);
    if (err != 0) return hip_failed(err);
    const ssm::LinChain ch{plan, a.out_slots, a.out_decay, h0, qk_dim * v_dim, 0};
    if ((err = ssm::launch_linattn_chain(ch, nullptr, stream)) != 0) return hip_failed(err);
    a.in_slots = a.out_slots;
  }
  a.out_seqs = h_final;
  a.out = o;
  err = z.bf16() ? ssm::launch_linattn_out_bf16(a, stream) : ssm::launch_linattn_out_f32(a, stream);
  if (err != 0) return hip_failed(err);
  if (zero_outside(c)) {
    ssm::LinZero r{};
    r.plan = plan;
    r.arrays[0] = {o, heads * v_dim * es};
    if ((err = ssm::launch_linattn_zero_outside(r, stream)) != 0) return hip_failed(err);
  }
  return ok();
}

int ssm_linattn_bwd_workspace_size(int64_t tokens, int64_t nseq, int packed, int64_t heads,
                                   int64_t qk_heads, int64_t qk_dim, int64_t v_dim, int dtype,
                                   int want_dg, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "bytes is NULL");
  if (want_dg < 0 || want_dg > 2) return fail(SSM_ERR_INVALID_ARG, "want_dg=%d: 0..2", want_dg);
  const Sizes z{tokens, nseq, heads, qk_heads, qk_dim, v_dim, dtype, packed != 0};
  int st = check_sizes(z);
  if (st != SSM_OK) return st;
  const ssm::LinPlan p = make_plan(z, true, want_dg != 0);
  if ((st = check_plan(z, p, want_dg ? 2 : 1)) != SSM_OK) return st;
  *bytes = static_cast<size_t>(bwd_layout(z, p, want_dg).total);
  return ok();
}

int ssm_linattn_bwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const float *g, unsigned flags, float scale,
                    const float *h0, const int32_t *cu_seqlens, const void *d_o,
                    const float *dh_final, void *dq, void *dk, void *dv, float *dg, float *dh0,
                    int64_t tokens, int64_t nseq, int64_t heads, int64_t qk_heads, int64_t qk_dim,
                    int64_t v_dim, int dtype, void *workspace, size_t workspace_bytes,
                    void *stream) {
  const Call c{{tokens, nseq, heads, qk_heads, qk_dim, v_dim, dtype, cu_seqlens != nullptr},
               q, k, v, q_stride, k_stride, v_stride, g, h0, cu_seqlens, flags, scale};
  int st = check_call(c, SSM_FLAG_HEAD_DECAY | SSM_FLAG_ZERO_OUTSIDE);
  if (st != SSM_OK) return st;
  const Sizes &z = c.z;
  const int64_t es = z.es();
  if (tokens > 0 && (!d_o || !dq || !dk || !dv))
    return fail(SSM_ERR_INVALID_ARG, "required pointer is NULL (d_o=%p dq=%p dk=%p dv=%p)", d_o,
                dq, dk, dv);
  if (dg && !g) return fail(SSM_ERR_INVALID_ARG, "dg without g");
  const void *acts[] = {d_o, dq, dk, dv};
  for (const void *p : acts)
    if (!aligned(p, es))
      return fail(SSM_ERR_INVALID_ARG, "activation pointer %p not %lld-byte aligned", p,
                  (long long)es);
  const void *words[] = {dh_final, dg, dh0};
  for (const void *p : words)
    if (!aligned(p, 4)) return fail(SSM_ERR_INVALID_ARG, "pointer %p not 4-byte aligned", p);
  const int want_dg = !dg ? 0 : flags & SSM_FLAG_HEAD_DECAY ? 2 : 1;
  ssm::LinPlan plan = make_plan(z, true, want_dg != 0);
  if ((st = check_plan(z, plan, want_dg ? 2 : 1)) != SSM_OK) return st;
  const BwdLayout l = bwd_layout(z, plan, want_dg);
  if ((st = check_workspace(workspace, workspace_bytes, static_cast<size_t>(l.total))) != SSM_OK)
    return st;
  const int64_t states = nseq * heads * qk_dim * v_dim * 4;
  const int64_t qk = tokens * qk_heads * qk_dim * es, vo = tokens * heads * v_dim * es;
  const Span ins[] = {{q, span_bytes(tokens, q_stride, qk_heads * qk_dim, es), "q"},
                      {k, span_bytes(tokens, k_stride, qk_heads * qk_dim, es), "k"},
                      {v, span_bytes(tokens, v_stride, heads * v_dim, es), "v"},
                      {g, g_bytes(c), "g"},
                      {h0, states, "h0"},
                      {cu_seqlens, (nseq + 1) * 4, "cu_seqlens"},
                      {d_o, vo, "d_o"},
                      {dh_final, states, "dh_final"}};
  const Span outs[] = {{dq, qk, "dq"}, {dk, qk, "dk"}, {dv, vo, "dv"}, {dg, g_bytes(c), "dg"},
                       {dh0, states, "dh0"}, {workspace, l.total, "workspace"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;

  plan.cu = cu_seqlens;
  const int64_t o_stride = heads * v_dim;
  plan.vec = rows16(q, q_stride, qk_dim, es) && rows16(k, k_stride, qk_dim, es) &&
             rows16(v, v_stride, v_dim, es) && rows16(d_o, o_stride, v_dim, es) &&
             aligned(dq, 16) && aligned(dk, 16) && aligned(dv, 16);
  const int64_t div = heads / qk_heads;
  const bool bf16 = z.bf16(), many = many_segments(z, plan);
  char *w = static_cast<char *>(workspace);
  auto f32 = [&](int64_t at) { return reinterpret_cast<float *>(w + at); };
  const ssm::LinSide Q = side(q, q_stride, qk_dim, div), K = side(k, k_stride, qk_dim, div);
  const ssm::LinSide V = side(v, v_stride, v_dim, 1), O = side(d_o, o_stride, v_dim, 1);
  int err;

  // S is stored (qk_dim, v_dim); so is its adjoint
  ssm::LinCore base{};
  base.plan = plan;
  base.g = g;
  base.g_kind = g_kind(c);
  if (many) {
    ssm::LinCore a = base;  // the states between segments
    a.q = K;
    a.k = K;
    a.v = V;
    a.into = 1.0f;
    a.sa = static_cast<int>(v_dim);
    a.sb = 1;
    a.out_slots = f32(l.states);
    a.out_decay = f32(l.decay);
    ssm::LinCore b = a;  // and their adjoints
    b.q = Q;
    b.k = Q;
    b.v = O;
    b.into = scale;
    b.out_slots = f32(l.adjoints);
    b.out_decay = f32(l.adecay);
    err = bf16 ? ssm::launch_linattn_states_bf16(a, &b, stream)
               : ssm::launch_linattn_states_f32(a, &b, stream);
    if (err != 0) return hip_failed(err);
    const ssm::LinChain fwd{plan, f32(l.states), f32(l.decay), h0, qk_dim * v_dim, 0};
    const ssm::LinChain rev{plan, f32(l.adjoints), f32(l.adecay), dh_final, qk_dim * v_dim, 1};
    if ((err = ssm::launch_linattn_chain(fwd, &rev, stream)) != 0) return hip_failed(err);
  }
  const bool shared = div > 1;
  ssm::LinCore gq = base;  // dq: in token order on S^T
  gq.q = O;
  gq.k = V;
  gq.v = K;
  gq.inter = gq.inside = scale;
  gq.into = 1.0f;
  gq.in_slots = many ? f32(l.states) : nullptr;
  gq.in_seqs = h0;
  gq.sa = 1;
  gq.sb = static_cast<int>(v_dim);
  gq.out = shared ? static_cast<void *>(f32(l.dq)) : dq;
  gq.out_f32 = shared;
  ssm::LinCore gk = gq;  // dk: against it on M^T
  gk.q = V;
  gk.k = O;
  gk.v = Q;
  gk.inter = 1.0f;
  gk.into = scale;
  gk.in_slots = many ? f32(l.adjoints) : nullptr;
  gk.in_seqs = dh_final;
  gk.out = shared ? static_cast<void *>(f32(l.dk)) : dk;
  ssm::LinCore gv = gk;  // dv: against it on M
  gv.q = K;
  gv.k = Q;
  gv.v = O;
  gv.sa = static_cast<int>(v_dim);
  gv.sb = 1;
  gv.out = dv;
  gv.out_f32 = 0;
  gv.out_seqs = dh0;
  if (want_dg) {
    gq.x = Q;
    gq.dots = f32(l.xdots);
    gq.out_seqs = f32(l.last);
    gk.x = K;
    gk.dots = f32(l.ydots);
  }
  const ssm::LinPairs pr{pairs_plan(z, plan), Q, K, V, O, g, base.g_kind, scale,
                         want_dg ? f32(l.pairs) : nullptr};
  err = bf16 ? ssm::launch_linattn_grads_bf16(gq, gk, gv, want_dg ? &pr : nullptr, stream)
             : ssm::launch_linattn_grads_f32(gq, gk, gv, want_dg ? &pr : nullptr, stream);
  if (err != 0) return hip_failed(err);
  if (shared && tokens > 0) {
    const int n = static_cast<int>(div), d = static_cast<int>(qk_dim);
    if ((err = ssm::launch_linattn_head_sum(f32(l.dq), f32(l.dk), dq, dk, plan, n, d, bf16,
                                            stream)) != 0)
      return hip_failed(err);
  }
  if (want_dg) {
    ssm::LinDecayGrad a{};
    a.plan = plan;
    a.pairs = f32(l.pairs);
    a.xdots = f32(l.xdots);
    a.ydots = f32(l.ydots);
    a.slices = static_cast<int>(slices_of(qk_dim));
    a.states = f32(l.states);
    a.adjoints = f32(l.adjoints);
    a.last = f32(l.last);
    a.dlast = dh_final;
    a.size = static_cast<int>(qk_dim * v_dim);
    a.g = g;
    a.g_kind = base.g_kind;
    a.chunk = ssm::linattn_chunk(bf16);
    a.dg = want_dg == 2 ? f32(l.dg) : dg;
    if ((err = ssm::launch_linattn_decay_grad(a, stream)) != 0) return hip_failed(err);
    if (want_dg == 2 &&
        (err = ssm::launch_linattn_token_sum(f32(l.dg), dg, plan, stream)) != 0)
      return hip_failed(err);
  }
  if (zero_outside(c)) {
    ssm::LinZero r{};
    r.plan = plan;
    r.arrays[0] = {dq, qk_heads * qk_dim * es};
    r.arrays[1] = {dk, qk_heads * qk_dim * es};
    r.arrays[2] = {dv, heads * v_dim * es};
    if (want_dg == 1) r.arrays[3] = {dg, heads * 4};
    if ((err = ssm::launch_linattn_zero_outside(r, stream)) != 0) return hip_failed(err);
  }
  return ok();
}

int ssm_linattn_step(float *state, const void *q, int64_t q_stride, const void *k,
                     int64_t k_stride, const void *v, int64_t v_stride, const float *g,
                     unsigned flags, float scale, const int32_t *slots, void *o, int64_t batch,
                     int64_t nslots, int64_t heads, int64_t qk_heads, int64_t qk_dim,
                     int64_t v_dim, int dtype, void *stream) {
  const Call c{{batch, 1, heads, qk_heads, qk_dim, v_dim, dtype, true},
               q, k, v, q_stride, k_stride, v_stride, g, nullptr, slots, flags, scale};
  int st = check_call(c, SSM_FLAG_HEAD_DECAY);
  if (st != SSM_OK) return st;
  const int64_t es = c.z.es();
  if (nslots <= 0 || nslots >= (int64_t(1) << 31))
    return fail(SSM_ERR_INVALID_ARG, "nslots=%lld out of range", (long long)nslots);
  if (!slots && batch > nslots)
    return fail(SSM_ERR_INVALID_ARG, "batch=%lld rows without slots, %lld states",
                (long long)batch, (long long)nslots);
  if (batch * heads * 4 > kMaxGroups)
    return fail(SSM_ERR_UNSUPPORTED, "batch=%lld heads=%lld: too many workgroups",
                (long long)batch, (long long)heads);
  if (batch == 0) return ok();
  if (!state || !o)
    return fail(SSM_ERR_INVALID_ARG, "required pointer is NULL (state=%p o=%p)", (void *)state, o);
  if (!aligned(state, 4) || !aligned(o, es))
    return fail(SSM_ERR_INVALID_ARG, "output not aligned (state=%p o=%p)", (void *)state, o);
  const Span ins[] = {{q, span_bytes(batch, q_stride, qk_heads * qk_dim, es), "q"},
                      {k, span_bytes(batch, k_stride, qk_heads * qk_dim, es), "k"},
                      {v, span_bytes(batch, v_stride, heads * v_dim, es), "v"},
                      {g, g_bytes(c), "g"},
                      {slots, batch * 4, "slots"}};
  const Span outs[] = {{state, nslots * heads * qk_dim * v_dim * 4, "state"},
                       {o, batch * heads * v_dim * es, "o"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;
  ssm::LinStep a{};
  a.state = state;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.g_kind = g_kind(c);
  a.slot_of = slots;
  a.o = o;
  a.scale = scale;
  a.batch = batch;
  a.slots = nslots;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.heads = static_cast<int>(heads);
  a.qk_heads = static_cast<int>(qk_heads);
  a.dk = static_cast<int>(qk_dim);
  a.dv = static_cast<int>(v_dim);
  const int err = ssm::launch_linattn_step(a, c.z.bf16(), stream);
  return err != 0 ? hip_failed(err) : ok();
}

}  // extern "C"

// ------------------------------------------------------------ block norm --
namespace {

struct NormCall {
  const void *x, *z, *residual;
  int64_t x_stride, z_stride, r_stride;
  const float *w_post, *scale, *w_pre;
  int64_t rows, dim, groups;
  float eps;
  int dtype, rdtype;
  int64_t es() const { return dtype == SSM_DTYPE_BF16 ? 2 : 4; }
  int64_t rs() const { return rdtype == SSM_DTYPE_BF16 ? 2 : 4; }
};

int check_norm_sizes(int64_t rows, int64_t dim, int64_t groups) {
  if (rows < 0 || dim <= 0 || groups <= 0)
    return fail(SSM_ERR_INVALID_ARG, "sizes out of range (rows=%lld dim=%lld groups=%lld)",
                (long long)rows, (long long)dim, (long long)groups);
  if (dim % groups != 0)
    return fail(SSM_ERR_INVALID_ARG, "dim=%lld is no multiple of groups=%lld", (long long)dim,
                (long long)groups);
  if (dim > ssm::kNormMaxDim || (groups > 1 && dim > ssm::kNormMaxDim / 2))
    return fail(SSM_ERR_UNSUPPORTED, "dim=%lld groups=%lld: this build supports dim up to %d, %d "
                "with groups", (long long)dim, (long long)groups, ssm::kNormMaxDim,
                ssm::kNormMaxDim / 2);
  // a workgroup a row, up to 1024 threads
  if (rows >= (int64_t(1) << 22))
    return fail(SSM_ERR_UNSUPPORTED, "rows=%lld: too many workgroups", (long long)rows);
  return SSM_OK;
}

int check_norm(const NormCall &c) {
  int st = check_norm_sizes(c.rows, c.dim, c.groups);
  if (st != SSM_OK) return st;
  if (c.dtype != SSM_DTYPE_F32 && c.dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_INVALID_ARG, "unknown dtype %d", c.dtype);
  if (c.rdtype != c.dtype && c.rdtype != SSM_DTYPE_F32)
    return fail(SSM_ERR_INVALID_ARG, "residual_dtype %d: the activations' or fp32", c.rdtype);
  if (!(c.eps > 0.0f) || !std::isfinite(c.eps))
    return fail(SSM_ERR_INVALID_ARG, "eps=%g must be positive", c.eps);
  if (c.rows > 0 && !c.x) return fail(SSM_ERR_INVALID_ARG, "x is NULL");
  if (c.groups > 1 && !c.w_post)
    return fail(SSM_ERR_INVALID_ARG, "groups=%lld without w_post", (long long)c.groups);
  if ((st = check_stride("x", c.x_stride, c.dim)) != SSM_OK) return st;
  if (c.z && (st = check_stride("z", c.z_stride, c.dim)) != SSM_OK) return st;
  if (c.residual && (st = check_stride("residual", c.r_stride, c.dim)) != SSM_OK) return st;
  if (!aligned(c.x, c.es()) || !aligned(c.z, c.es()) || !aligned(c.residual, c.rs()))
    return fail(SSM_ERR_INVALID_ARG, "activation pointer not aligned");
  if (!aligned(c.w_post, 4) || !aligned(c.scale, 4) || !aligned(c.w_pre, 4))
    return fail(SSM_ERR_INVALID_ARG, "weights not 4-byte aligned");
  return SSM_OK;
}

ssm::NormArgs norm_args(const NormCall &c) {
  ssm::NormArgs a{};
  a.x = c.x;
  a.z = c.z;
  a.residual = c.residual;
  a.w_post = c.w_post;
  a.scale = c.scale;
  a.w_pre = c.w_pre;
  a.x_stride = c.x_stride;
  a.z_stride = c.z_stride;
  a.r_stride = c.r_stride;
  a.rows = c.rows;
  a.dim = static_cast<int>(c.dim);
  a.groups = static_cast<int>(c.groups);
  a.eps = c.eps;
  a.wide = c.dtype == SSM_DTYPE_BF16 && c.rdtype == SSM_DTYPE_F32;
  return a;
}

// Whole 16-byte pieces: rows (and the pieces in fp32) start on 16 bytes.
bool norm_vec(const NormCall &c, const void *const *dense, int n) {
  if (c.dim * c.es() % 16 != 0) return false;
  if (!rows16(c.x, c.x_stride, c.dim, c.es())) return false;
  if (c.z && !rows16(c.z, c.z_stride, c.dim, c.es())) return false;
  if (c.residual && !rows16(c.residual, c.r_stride, c.dim, c.rs())) return false;
  if (!aligned(c.w_post, 16) || !aligned(c.scale, 16) || !aligned(c.w_pre, 16)) return false;
  for (int i = 0; i < n; ++i)
    if (!aligned(dense[i], 16)) return false;
  return true;
}

}  // namespace

extern "C" {

int ssm_block_norm_fwd(const void *x, int64_t x_stride, const float *w_post, const void *z,
                       int64_t z_stride, const float *scale, const void *residual,
                       int64_t residual_stride, const float *w_pre, void *r, void *y,
                       int64_t rows, int64_t dim, int64_t groups, float eps, int dtype,
                       int residual_dtype, void *stream) {
  const NormCall c{x, z, residual, x_stride, z_stride, residual_stride, w_post, scale, w_pre,
                   rows, dim, groups, eps, dtype, residual_dtype};
  int st = check_norm(c);
  if (st != SSM_OK) return st;
  if (rows == 0) return ok();
  if ((y != nullptr) != (w_pre != nullptr))
    return fail(SSM_ERR_INVALID_ARG, "y and w_pre go together");
  if (!r && !y) return fail(SSM_ERR_INVALID_ARG, "r is NULL and there is no y");
  if (!aligned(r, c.rs()) || !aligned(y, c.es()))
    return fail(SSM_ERR_INVALID_ARG, "output not aligned (r=%p y=%p)", r, y);
  const bool in_place = r && r == residual && residual_stride == dim;
  const Span ins[] = {{x, span_bytes(rows, x_stride, dim, c.es()), "x"},
                      {z, span_bytes(rows, z_stride, dim, c.es()), "z"},
                      {w_post, dim * 4, "w_post"}, {scale, dim * 4, "scale"},
                      {w_pre, dim * 4, "w_pre"},
                      {in_place ? nullptr : residual,
                       span_bytes(rows, residual_stride, dim, c.rs()), "residual"}};
  const Span outs[] = {{r, rows * dim * c.rs(), "r"}, {y, rows * dim * c.es(), "y"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;
  ssm::NormArgs a = norm_args(c);
  a.r = r;
  a.y = y;
  const void *dense[] = {r, y};
  a.vec = norm_vec(c, dense, 2);
  const int err = ssm::launch_block_norm_fwd(a, dtype == SSM_DTYPE_BF16, stream);
  return err != 0 ? hip_failed(err) : ok();
}

int ssm_block_norm_bwd_workspace_size(int64_t rows, int64_t dim, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "bytes is NULL");
  const int st = check_norm_sizes(rows, dim, 1);
  if (st != SSM_OK) return st;
  *bytes = static_cast<size_t>(ssm::norm_parts(rows)) * 3 * dim * 4;
  return ok();
}

int ssm_block_norm_bwd(const void *x, int64_t x_stride, const float *w_post, const void *z,
                       int64_t z_stride, const float *scale, const void *residual,
                       int64_t residual_stride, const float *w_pre, const void *dr,
                       const void *dy, void *dx, float *dw_post, void *dz, float *dscale,
                       void *dresidual, float *dw_pre, int64_t rows, int64_t dim, int64_t groups,
                       float eps, int dtype, int residual_dtype, void *workspace,
                       size_t workspace_bytes, void *stream) {
  const NormCall c{x, z, residual, x_stride, z_stride, residual_stride, w_post, scale, w_pre,
                   rows, dim, groups, eps, dtype, residual_dtype};
  int st = check_norm(c);
  if (st != SSM_OK) return st;
  if ((dw_post && !w_post) || (dz && !z) || (dscale && !scale) || (dresidual && !residual) ||
      (dw_pre && !w_pre))
    return fail(SSM_ERR_INVALID_ARG, "a gradient is given for an input that is not");
  if (rows > 0 && (dy != nullptr) != (w_pre != nullptr))
    return fail(SSM_ERR_INVALID_ARG, "dy and w_pre go together");
  if (rows > 0 && !dx) return fail(SSM_ERR_INVALID_ARG, "dx is NULL");
  if (!aligned(dr, c.rs()) || !aligned(dresidual, c.rs()) || !aligned(dy, c.es()) ||
      !aligned(dx, c.es()) || !aligned(dz, c.es()))
    return fail(SSM_ERR_INVALID_ARG, "activation pointer not aligned");
  if (!aligned(dw_post, 4) || !aligned(dscale, 4) || !aligned(dw_pre, 4))
    return fail(SSM_ERR_INVALID_ARG, "weight gradients not 4-byte aligned");
  const int64_t need = static_cast<int64_t>(ssm::norm_parts(rows)) * 3 * dim * 4;
  if ((st = check_workspace(workspace, workspace_bytes, static_cast<size_t>(need))) != SSM_OK)
    return st;
  const int64_t act = rows * dim * c.es(), wide = rows * dim * c.rs();
  const Span ins[] = {{x, span_bytes(rows, x_stride, dim, c.es()), "x"},
                      {z, span_bytes(rows, z_stride, dim, c.es()), "z"},
                      {w_post, dim * 4, "w_post"}, {scale, dim * 4, "scale"},
                      {w_pre, dim * 4, "w_pre"},
                      {residual, span_bytes(rows, residual_stride, dim, c.rs()), "residual"},
                      {dr, wide, "dr"}, {dy, act, "dy"}};
  const Span outs[] = {{dx, act, "dx"}, {dz, act, "dz"}, {dresidual, wide, "dresidual"},
                       {dw_post, dim * 4, "dw_post"}, {dscale, dim * 4, "dscale"},
                       {dw_pre, dim * 4, "dw_pre"}, {workspace, need, "workspace"}};
  if ((st = check_overlaps(ins, outs)) != SSM_OK) return st;
  ssm::NormArgs a = norm_args(c);
  a.dr = dr;
  a.dy = dy;
  a.dx = dx;
  a.dz = dz;
  a.dresidual = dresidual;
  a.dw_post = dw_post;
  a.dscale = dscale;
  a.dw_pre = dw_pre;
  a.parts = static_cast<float *>(workspace);
  a.nparts = ssm::norm_parts(rows);
  const void *dense[] = {dr, dy, dx, dz, dresidual, dw_post, dscale, dw_pre};
  a.vec = norm_vec(c, dense, 8);
  const int err = ssm::launch_block_norm_bwd(a, dtype == SSM_DTYPE_BF16, stream);
  return err != 0 ? hip_failed(err) : ok();
}

}  // extern "C"
