/*
 * moe_expert_w4.h -- C ABI of the experts' product with 4-bit weights in
 * libmoe_route.so: a serving form of moe_expert_gemm for batches that are bound
 * by the bytes of the weights.
 *
 * "Lower latency and higher throughput with multi-node DeepSeek deployment",
 * section "Quantization" (weights in few bits with scales per block); the
 * product stands between dispatch and combine like those of moe_expert.h,
 * whose conventions hold here: dims and expert_offsets, rows outside the
 * groups untouched, sums in f32 in parts, results that overlap other arrays
 * refused, nothing allocated, any call capturable.
 */
#ifndef MOE_EXPERT_W4_H
#define MOE_EXPERT_W4_H

#include "moe_expert.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Product of each expert's rows with its matrix of 4-bit weights,
 *   w[e][f][k] = row_scales[e][f] * group_scales[e][k/group][f] * q[e][f][k].
 *   group        32, 64 or 128; K % group == 0
 *   x            bf16 [N*cap][K]
 *   wq           i32 [E][W][K/8], W = F (linear) or 2F (gated: gate rows, then up
 *                rows): word i of a row holds elements 8i to 8i + 7 as 4-bit two's
 *                complement q in [-8, 7], element 8i + 2j at bit 4j and element
 *                8i + 2j + 1 at bit 16 + 4j (j = 0..3)
 *   group_scales e4m3 [E][K/group][W]: rows of a group next to each other
 *   row_scales   f32 [E][W]
 *   act MOE_EXPERT_LINEAR: y [N*cap][F] of dims->y_dtype
 *   act MOE_EXPERT_SWIGLU: y bf16 [N*cap][F] = silu(g) * u, whatever dims->y_dtype
 * q times its group's scale has at most seven significant bits and is
 * multiplied by x exactly; a row's scale multiplies the f32 sum.  x and wq must
 * be 16-byte aligned, y too, group_scales 8-byte, row_scales 4-byte.  With N = E = R = 1
 * (expert_offsets = {0, T}, cap_rows = T) this is the product of a dense layer,
 * for T = 1 a matrix-vector product. */
int moe_expert_gemm_w4(const MoeDims *dims, int K, int F, int act, int group, const void *x, const int32_t *wq,
                       const void *group_scales, const float *row_scales, const int32_t *expert_offsets, void *y,
                       void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERT_W4_H */
