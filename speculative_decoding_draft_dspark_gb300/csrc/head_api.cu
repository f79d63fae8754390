// C entry points of include/dspark_head.h: host-side validation, then the
// launches.  Nothing here allocates device memory or synchronises.
#include <cmath>
#include <cstdint>

#include "head_internal.h"

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

}  // extern "C"
