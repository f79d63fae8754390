// Internal interfaces between the C-ABI layer (head_api.cu) and the kernels
// that train the drafter's head (head_loss.cu, norm.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/dspark_head.h"
#include "dspark_internal.h"

namespace dspark {

// ------------------------------------------------------------------ loss
// Where the pieces of a head workspace lie (bytes from its base).  Everything
// but the status word is scratch of one call.
struct HeadLayout {
  int64_t rows_pad;   // M rounded up to the 256 rows of a tile
  int64_t cols_pad;   // d and rank, each rounded up to 64, together
  int64_t piece;      // vocabulary entries handled at a time by the gradient
  int32_t splits;     // partial sums of the gradient of [h, U[prev]]
  size_t rowinfo;     // per counted row: index, target, prev, lse, weight, z_t
  size_t a;           // bf16 [rows_pad, cols_pad]: [h, U[prev]]
  size_t partial;     // loss: float2 [epilogue warps][rows_pad] (max, sum)
  size_t g;           // gradient: G^T, bf16 [piece, rows_pad]
  size_t acc;         // gradient: sums of dA^T, fp32 [splits][cols_pad][rows_pad]
  size_t de;          // gradient: fp32 [rows_pad, rank], dA's tail by rows
  size_t total;
};
HeadLayout head_layout(int32_t M, int32_t vocab, int32_t d, int32_t rank, bool grad);

struct HeadArgs {
  const void *h;
  int64_t h_stride;
  const void *W, *U, *V;
  const int32_t *prev, *target;
  int32_t M, vocab, d, rank;
  float *loss, *lse;         // loss: outputs; gradient: lse is an input
  const float *dloss;        // gradient only, as what follows
  void *dh;
  int64_t dh_stride;
  void *dW, *dU, *dV;
  uint8_t *workspace;
};
dspark_status head_loss_launch(const HeadArgs &a, cudaStream_t stream);
dspark_status head_loss_grad_launch(const HeadArgs &a, cudaStream_t stream);

}  // namespace dspark
