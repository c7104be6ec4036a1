// ssm_model_internal.h -- launch interface of the embedding, the layer norm
// and the gradients' norm (ssm_embed.hip, ssm_layer_norm.hip, ssm_grad.hip).
// Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ssm {

// ------------------------------------------------------------- embedding --
constexpr int kEmbedMaxDim = 65536;

struct EmbedArgs {
  const void *ids;
  int wide_ids;  // int64
  int64_t tokens, vocab;
  int dim;
  float scale;
  // forward
  const void *weight;
  int64_t w_stride;
  void *out;
  // backward
  const void *dy;
  int64_t dy_stride;
  void *dweight;
  int accumulate;
  void *workspace;
};

int64_t embed_bwd_workspace(int64_t tokens, int64_t dim);
// w_bf16: of weight or dweight; bf16: of out or dy
int launch_embed_fwd(const EmbedArgs &a, bool w_bf16, bool bf16, void *stream);
int launch_embed_bwd(const EmbedArgs &a, bool w_bf16, bool bf16, void *stream);

// ------------------------------------------------------------ layer norm --
constexpr int kLayerNormMaxDim = 16384;

struct LayerNormArgs {
  const void *x, *residual;
  int64_t x_stride, r_stride;
  const float *weight, *bias;
  int64_t rows;
  int dim;
  float eps;
  // forward
  void *r, *y;
  // backward
  const void *dr, *dy;
  void *dx, *dresidual;
  float *dweight, *dbias;
  float *parts;  // (workgroups, 2, dim)
  int nparts;
};

enum LayerNormTypes { kLnBf16 = 0, kLnBf16Wide = 1, kLnF32 = 2, kLnF32Bf16 = 3 };

// Workgroups of the backward pass, and partial rows of the weights' gradients,
// at most, for any types.
int layer_norm_bwd_parts(int64_t rows, int dim);
int launch_layer_norm_fwd(const LayerNormArgs &a, LayerNormTypes types, void *stream);
int launch_layer_norm_bwd(const LayerNormArgs &a, LayerNormTypes types, void *stream);

// -------------------------------------------------------- gradients' norm --
constexpr int kGradTensors = 160;   // tensors a launch takes, in its arguments
constexpr int kGradGroups = 2048;   // most workgroups that sum squares, and their sums
constexpr int kGradChunk = 16384;   // elements that a workgroup takes at a time
constexpr int64_t kGradPiece = int64_t(1) << 29;  // elements of an entry; longer tensors have several

constexpr int kGradSmall = 8192;    // most pieces of 8 elements that one workgroup takes alone

struct GradTable {
  const void *grad[kGradTensors];
  uint32_t first[kGradTensors + 1];  // chunks (or pieces) before each entry
  // elements of each entry; its gradient's and its output's types
  uint32_t size[kGradTensors];
  int32_t n;
};
constexpr uint32_t kGradBf16 = 1u << 31, kGradOutBf16 = 1u << 30;
constexpr uint32_t kGradSize = kGradOutBf16 - 1;

struct GradOuts {
  void *out[kGradTensors];
};

// Norm and (with clip) clipping of a table that counts pieces.
int launch_grad_small(const GradTable &t, const GradOuts &outs, bool clip, bool in_place,
                      float max_norm, float *norm, void *stream);
// Adds the squares of a table's tensors to nsums (at most kGradGroups) sums,
// or writes them where it is the first.
int launch_grad_squares(const GradTable &t, double *sums, int nsums, bool first, void *stream);
int launch_grad_norm(const double *sums, int nsums, float *norm, void *stream);
// sums: null where norm is given
int launch_grad_scale(const GradTable &t, const GradOuts &outs, bool in_place,
                      const double *sums, int nsums, float max_norm, float *norm, bool write_norm,
                      void *stream);

}  // namespace ssm
