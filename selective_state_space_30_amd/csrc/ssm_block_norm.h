// ssm_block_norm.h -- launch interface of the block norm (ssm_block_norm.hip).
// Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ssm {

constexpr int kNormMaxDim = 16384;
constexpr int kNormMaxParts = 1024;  // workgroups that leave partial weight gradients

struct NormArgs {
  const void *x, *z, *residual;       // residual: fp32 if wide, else the activations' type
  const float *w_post, *scale, *w_pre;
  int64_t x_stride, z_stride, r_stride;
  int64_t rows;
  int dim, groups;
  float eps;
  int wide;                           // residual, r (and their gradients) in fp32
  // forward
  void *r, *y;
  // backward
  const void *dr, *dy;                // nullable gradients of r and y
  void *dx, *dz, *dresidual;
  float *dw_post, *dscale, *dw_pre;
  float *parts;                       // (workgroups, 3, dim)
  int nparts;
  int vec;                            // rows are read and written in 16-byte pieces
};

// workgroups of the backward pass
int norm_parts(int64_t rows);
int launch_block_norm_fwd(const NormArgs &a, bool bf16, void *stream);
int launch_block_norm_bwd(const NormArgs &a, bool bf16, void *stream);

}  // namespace ssm
