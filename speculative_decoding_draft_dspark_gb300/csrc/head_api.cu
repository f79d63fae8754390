// C entry points of include/dspark_head.h: host-side validation, then the
// launches.  Nothing here allocates device memory or synchronises.
#include <cmath>
#include <cstdint>

#include "head_internal.h"
#include "norm_internal.h"

namespace dspark {
namespace {

bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

dspark_status check_head_dims(int32_t M, int32_t vocab, int32_t d, int32_t rank) {
  if (M <= 0 || vocab <= 0 || d <= 0 || rank < 0) return DSPARK_ERR_INVALID_ARG;
  if (M > (1 << 20) || vocab >= (1 << 30)) return DSPARK_ERR_UNSUPPORTED;
  if (d % 8 != 0 || d > 65536) return DSPARK_ERR_UNSUPPORTED;
  if (rank % 8 != 0 || rank > 256) return DSPARK_ERR_UNSUPPORTED;
  // tiles of 256 x 256 are counted in 32 bits
  const int64_t tiles = ((static_cast<int64_t>(M) + 255) / 256) *
                        ((static_cast<int64_t>(vocab) + 255) / 256);
  if (tiles > (1ll << 30)) return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

dspark_status check_head_inputs(const void *h, int64_t h_stride, const void *W, const void *U,
                                const void *V, const int32_t *prev, const int32_t *target,
                                const float *lse, int32_t M, int32_t vocab, int32_t d,
                                int32_t rank) {
  const dspark_status s = check_head_dims(M, vocab, d, rank);
  if (s != DSPARK_OK) return s;
  if (!h || !W || !target || !lse) return DSPARK_ERR_INVALID_ARG;
  if (rank > 0 && (!U || !V || !prev)) return DSPARK_ERR_INVALID_ARG;
  if (h_stride < d || h_stride % 8 != 0) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(target, 4) || !aligned(lse, 4))
    return DSPARK_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned(U, 16) || !aligned(V, 16) || !aligned(prev, 4)))
    return DSPARK_ERR_INVALID_ARG;
  return DSPARK_OK;
}

dspark_status check_head_ws(const void *ws, size_t bytes, int32_t M, int32_t vocab, int32_t d,
                            int32_t rank, bool grad) {
  if (ws == nullptr || !aligned(ws, 256) || bytes < head_layout(M, vocab, d, rank, grad).total)
    return DSPARK_ERR_WORKSPACE;
  return DSPARK_OK;
}

// A [M, d] tensor's pointer and row stride; `need`: it may not be NULL.
bool rows_ok(const void *p, int64_t stride, int32_t d, int esz, bool need) {
  if (p == nullptr) return !need;
  return stride >= d && aligned(p, esz);
}

dspark_status check_norm_dims(int32_t dtype, int32_t M, int32_t d, float p) {
  if (dtype != DSPARK_BF16 && dtype != DSPARK_F32) return DSPARK_ERR_INVALID_ARG;
  if (M <= 0 || d <= 0) return DSPARK_ERR_INVALID_ARG;
  if (!(p >= 0.0f && p <= 1.0f)) return DSPARK_ERR_INVALID_ARG;
  if (d > kMaxNormColumns || M > (1 << 30)) return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

DropArgs drop_args(float p, uint64_t seed, uint32_t offset) {
  DropArgs a = {};
  const double keep = std::floor((1.0 - static_cast<double>(p)) * 65536.0 + 0.5);
  a.on = keep < 65536.0;
  a.keep_hi = static_cast<uint32_t>(keep) << 16;
  a.scale = keep > 0.0 ? static_cast<float>(65536.0 / keep) : 0.0f;
  a.seed_lo = static_cast<uint32_t>(seed);
  a.seed_hi = static_cast<uint32_t>(seed >> 32);
  a.offset = offset;
  return a;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

size_t dspark_head_workspace_size(int32_t M, int32_t vocab, int32_t d, int32_t rank,
                                  int32_t grad) {
  if (check_head_dims(M, vocab, d, rank) != DSPARK_OK) return 0;
  const size_t loss = head_layout(M, vocab, d, rank, false).total;
  if (!grad) return loss;
  const size_t both = head_layout(M, vocab, d, rank, true).total;
  return both > loss ? both : loss;
}

dspark_status dspark_head_loss(const void *h, int64_t h_stride, const void *W, const void *U,
                               const void *V, const int32_t *prev, const int32_t *target,
                               int32_t M, int32_t vocab, int32_t d, int32_t rank, float *loss,
                               float *lse, void *workspace, size_t workspace_bytes,
                               dspark_stream_t stream) {
  dspark_status s =
      check_head_inputs(h, h_stride, W, U, V, prev, target, lse, M, vocab, d, rank);
  if (s != DSPARK_OK) return s;
  if (!loss || !aligned(loss, 4)) return DSPARK_ERR_INVALID_ARG;
  if ((s = check_head_ws(workspace, workspace_bytes, M, vocab, d, rank, false)) != DSPARK_OK)
    return s;
  HeadArgs a = {};
  a.h = h;
  a.h_stride = h_stride;
  a.W = W;
  a.U = U;
  a.V = V;
  a.prev = prev;
  a.target = target;
  a.M = M;
  a.vocab = vocab;
  a.d = d;
  a.rank = rank;
  a.loss = loss;
  a.lse = lse;
  a.workspace = static_cast<uint8_t *>(workspace);
  return head_loss_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

dspark_status dspark_head_loss_grad(const void *h, int64_t h_stride, const void *W, const void *U,
                                    const void *V, const int32_t *prev, const int32_t *target,
                                    const float *lse, const float *dloss, int32_t M,
                                    int32_t vocab, int32_t d, int32_t rank, void *dh,
                                    int64_t dh_stride, void *dW, void *dU, void *dV,
                                    void *workspace, size_t workspace_bytes,
                                    dspark_stream_t stream) {
  dspark_status s =
      check_head_inputs(h, h_stride, W, U, V, prev, target, lse, M, vocab, d, rank);
  if (s != DSPARK_OK) return s;
  if (!dloss || !aligned(dloss, 4) || !dh || !aligned(dh, 16) || !dW || !aligned(dW, 16))
    return DSPARK_ERR_INVALID_ARG;
  if (dh_stride < d || dh_stride % 8 != 0) return DSPARK_ERR_INVALID_ARG;
  if (rank > 0 && (!dU || !dV || !aligned(dU, 16) || !aligned(dV, 16)))
    return DSPARK_ERR_INVALID_ARG;
  if ((s = check_head_ws(workspace, workspace_bytes, M, vocab, d, rank, true)) != DSPARK_OK)
    return s;
  HeadArgs a = {};
  a.h = h;
  a.h_stride = h_stride;
  a.W = W;
  a.U = U;
  a.V = V;
  a.prev = prev;
  a.target = target;
  a.M = M;
  a.vocab = vocab;
  a.d = d;
  a.rank = rank;
  a.lse = const_cast<float *>(lse);
  a.dloss = dloss;
  a.dh = dh;
  a.dh_stride = dh_stride;
  a.dW = dW;
  a.dU = dU;
  a.dV = dV;
  a.workspace = static_cast<uint8_t *>(workspace);
  return head_loss_grad_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

dspark_status dspark_residual_norm(const void *x, int64_t x_stride, const void *residual,
                                   int64_t residual_stride, const void *gain, int32_t dtype,
                                   int32_t M, int32_t d, float eps, float p, uint64_t seed,
                                   uint32_t offset, void *r, int64_t r_stride, void *y,
                                   int64_t y_stride, int32_t y_dtype, int32_t group,
                                   float *scale, float *rstd, dspark_stream_t stream) {
  const dspark_status s = check_norm_dims(dtype, M, d, p);
  if (s != DSPARK_OK) return s;
  const int e = dtype == DSPARK_F32 ? 4 : 2;
  const bool e4m3 = y_dtype == DSPARK_E4M3;
  if (!e4m3 && y_dtype != dtype) return DSPARK_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return DSPARK_ERR_INVALID_ARG;
  if (!rows_ok(x, x_stride, d, e, true) || !rows_ok(residual, residual_stride, d, e, false) ||
      !rows_ok(r, r_stride, d, e, false) || !rows_ok(y, y_stride, d, e4m3 ? 1 : e, true) ||
      !rows_ok(gain, d, d, e, true) || (rstd && !aligned(rstd, 4)))
    return DSPARK_ERR_INVALID_ARG;
  if (e4m3) {
    if (group != 0 && group != 128) return DSPARK_ERR_UNSUPPORTED;
    if (!scale || !aligned(scale, 4)) return DSPARK_ERR_INVALID_ARG;
  }
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.gain = gain;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.f32 = dtype == DSPARK_F32;
  a.M = M;
  a.d = d;
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(d);
  a.drop = drop_args(p, seed, offset);
  a.r = r;
  a.y = y;
  a.r_stride = r_stride;
  a.y_stride = y_stride;
  a.e4m3 = e4m3;
  a.group = group;
  a.groups = group ? (d + group - 1) / group : 1;
  a.scale = scale;
  a.rstd = rstd;
  return norm_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t dspark_norm_workspace_size(int32_t M, int32_t d) {
  if (check_norm_dims(DSPARK_BF16, M, d, 0.0f) != DSPARK_OK) return 0;
  return norm_workspace_bytes(M, d);
}

dspark_status dspark_residual_norm_grad(const void *dy, int64_t dy_stride, const void *dr,
                                        int64_t dr_stride, const void *r, int64_t r_stride,
                                        const void *gain, const float *rstd, int32_t dtype,
                                        int32_t M, int32_t d, float p, uint64_t seed,
                                        uint32_t offset, void *dx, int64_t dx_stride,
                                        void *dresidual, int64_t dresidual_stride, void *dgain,
                                        void *workspace, size_t workspace_bytes,
                                        dspark_stream_t stream) {
  const dspark_status s = check_norm_dims(dtype, M, d, p);
  if (s != DSPARK_OK) return s;
  const int e = dtype == DSPARK_F32 ? 4 : 2;
  if (!rows_ok(dy, dy_stride, d, e, true) || !rows_ok(dr, dr_stride, d, e, false) ||
      !rows_ok(r, r_stride, d, e, true) || !rows_ok(gain, d, d, e, true) ||
      !rows_ok(dx, dx_stride, d, e, false) ||
      !rows_ok(dresidual, dresidual_stride, d, e, false) || !rows_ok(dgain, d, d, e, false) ||
      !rstd || !aligned(rstd, 4))
    return DSPARK_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < norm_workspace_bytes(M, d))
    return DSPARK_ERR_WORKSPACE;
  NormGradArgs a = {};
  a.dy = dy;
  a.dr = dr;
  a.r = r;
  a.gain = gain;
  a.dy_stride = dy_stride;
  a.dr_stride = dr_stride;
  a.r_stride = r_stride;
  a.rstd = rstd;
  a.f32 = dtype == DSPARK_F32;
  a.M = M;
  a.d = d;
  a.inv_d = 1.0f / static_cast<float>(d);
  a.drop = drop_args(p, seed, offset);
  a.dx = dx;
  a.dresidual = dresidual;
  a.dgain = dgain;
  a.dx_stride = dx_stride;
  a.dresidual_stride = dresidual_stride;
  a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kNormPartialOffset);
  return norm_grad_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

dspark_status dspark_dropout(const void *x, int64_t x_stride, const void *residual,
                             int64_t residual_stride, int32_t dtype, int32_t M, int32_t d,
                             float p, uint64_t seed, uint32_t offset, void *y, int64_t y_stride,
                             dspark_stream_t stream) {
  const dspark_status s = check_norm_dims(dtype, M, d, p);
  if (s != DSPARK_OK) return s;
  const int e = dtype == DSPARK_F32 ? 4 : 2;
  if (!rows_ok(x, x_stride, d, e, true) || !rows_ok(residual, residual_stride, d, e, false) ||
      !rows_ok(y, y_stride, d, e, true))
    return DSPARK_ERR_INVALID_ARG;
  DropoutArgs a = {};
  a.x = x;
  a.residual = residual;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.f32 = dtype == DSPARK_F32;
  a.M = M;
  a.d = d;
  a.drop = drop_args(p, seed, offset);
  a.y = y;
  a.y_stride = y_stride;
  return dropout_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
