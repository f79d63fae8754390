// Internal interface between the C-ABI layer (head_api.cu) and norm.cu.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/dspark_head.h"

namespace dspark {

struct DropArgs {
  int32_t on;         // something is dropped
  uint32_t keep_hi;   // T 65536: kept iff the 16-bit lane, in a word's upper half, is below
  float scale;        // 65536 / T
  uint32_t seed_lo, seed_hi, offset;
};

struct NormArgs {
  const void *x, *residual, *gain;
  int64_t x_stride, residual_stride;  // elements
  int32_t f32, M, d;
  float eps, inv_d;
  DropArgs drop;
  void *r, *y;
  int64_t r_stride, y_stride;
  int32_t e4m3, group, groups;  // group 0: a scale for the row; groups: scales a row
  float *scale, *rstd;
};

struct NormGradArgs {
  const void *dy, *dr, *r, *gain;
  int64_t dy_stride, dr_stride, r_stride;
  const float *rstd;
  int32_t f32, M, d;
  float inv_d;
  DropArgs drop;
  void *dx, *dresidual, *dgain;
  int64_t dx_stride, dresidual_stride;
  float *partial;
};

struct DropoutArgs {
  const void *x, *residual;
  int64_t x_stride, residual_stride;
  int32_t f32, M, d;
  DropArgs drop;
  void *y;
  int64_t y_stride;
};

constexpr int kMaxNormColumns = 32768;
constexpr size_t kNormPartialOffset = 256;
size_t norm_workspace_bytes(int32_t M, int32_t d);
dspark_status norm_launch(const NormArgs &a, cudaStream_t stream);
dspark_status norm_grad_launch(const NormGradArgs &a, cudaStream_t stream);
dspark_status dropout_launch(const DropoutArgs &a, cudaStream_t stream);

}  // namespace dspark
