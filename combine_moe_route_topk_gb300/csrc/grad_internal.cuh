// Launchers of the routing steps' gradients (arguments already validated).
#pragma once

#include "moe_grad.h"
#include "moe_internal.cuh"

namespace moe {

cudaError_t launch_combine_grad(const void *dout, const void *y, int y_dtype, const int32_t *pos, const float *topk_w,
                                int64_t NT, int R, int H, int64_t rows_total, void *dy, float *dtopk_w,
                                cudaStream_t stream);
cudaError_t launch_dispatch_grad(const void *dpacked, int x_dtype, const int32_t *pos, const void *add, int64_t NT,
                                 int R, int H, int64_t rows_total, void *dx, cudaStream_t stream);
cudaError_t launch_route_grad(const float *logits, const float *bias, int64_t NT, int E, int R, int score_fn,
                              int renormalize, const int32_t *topk_idx, const float *topk_w, const float *dtopk_w,
                              float *dlogits, float *dbias, cudaStream_t stream);

}  // namespace moe
