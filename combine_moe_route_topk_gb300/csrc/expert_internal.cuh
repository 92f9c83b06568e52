// Launchers of the experts' products (arguments already validated).
#pragma once

#include "moe_expert.h"
#include "moe_internal.cuh"

namespace moe {

// Where the experts' rows are.
struct ExpertRows {
    const int32_t *offsets;  // device, [E + 1]
    int E, L;                // experts, experts per rank
    int64_t cap, rows_total;  // rows of a region, of all of them
    int64_t most, pairs;      // rows that one expert can have, that all of them can
};

cudaError_t launch_expert_gemm(const ExpertRows &r, int K, int F, int gated, const void *x, const void *w, void *y,
                               int y_f32, void *pre, cudaStream_t stream);
cudaError_t launch_expert_dgrad(const ExpertRows &r, int K, int F, const void *dy, const void *w, void *dx,
                                cudaStream_t stream);
cudaError_t launch_expert_wgrad(const ExpertRows &r, int K, int F, const void *dy, const void *x, void *dw, int dw_f32,
                                cudaStream_t stream);
cudaError_t launch_expert_swiglu_grad(const ExpertRows &r, int N, int64_t pairs, int F, const void *pre, const void *dh,
                                      void *dpre, cudaStream_t stream);
cudaError_t launch_expert_gemm_fp8(const ExpertRows &r, int K, int F, int gated, const void *xq, const float *x_scales,
                                   const void *wq, const float *w_scales, void *y, int y_f32, float *y_scales,
                                   cudaStream_t stream);

// Read and clear the error words of the kernels above (set when a bounded
// wait gave up); the caller has waited for the stream.
cudaError_t take_expert_gemm_error(int *err);
cudaError_t take_expert_wgrad_error(int *err);
cudaError_t take_expert_fp8_error(int *err);

}  // namespace moe
