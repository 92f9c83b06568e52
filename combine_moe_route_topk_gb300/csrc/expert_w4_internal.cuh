// Launcher of the experts' product with 4-bit weights (arguments already validated).
#pragma once

#include "expert_internal.cuh"
#include "moe_expert_w4.h"

namespace moe {

cudaError_t launch_expert_gemm_w4(const ExpertRows &r, int K, int F, int gated, int group, const void *x,
                                  const void *wq, const void *group_scales, const float *row_scales, void *y, int y_f32,
                                  cudaStream_t stream);
cudaError_t take_expert_w4_error(int *err);

// The form for experts with few rows.
cudaError_t launch_expert_w4_few(const ExpertRows &r, int K, int F, int gated, int group, const void *x, const void *wq,
                                 const void *group_scales, const float *row_scales, void *y, int y_f32,
                                 cudaStream_t stream);
cudaError_t take_expert_w4_few_error(int *err);

}  // namespace moe
