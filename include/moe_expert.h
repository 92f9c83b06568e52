/*
 * moe_expert.h -- C ABI of the experts' products in libmoe_route.so: what a
 * Mixture-of-Experts layer computes between dispatch and combine, on the
 * receive layout that moe_dispatch_count defines and the packs write.
 *
 * "Lower latency and higher throughput with multi-node DeepSeek deployment",
 * section "Computation and communication overlap" (the grouped product runs
 * between dispatch and combine) and section "Quantization" (fp8 operands with
 * block scales); "Efficient and portable mixture-of-experts communication",
 * section "Dispatch" (tokens grouped per expert for the grouped product).
 *
 * The conventions of moe_route.h hold: device pointers owned by the caller,
 * dense row-major arrays, work enqueued on `stream`, no host
 * synchronisation, nothing allocated and no workspace, grids that do not
 * depend on routing (every call can be captured in a CUDA graph, and calls
 * may overlap as long as their outputs do not), argument errors reported
 * before anything is enqueued.  More precisely:
 *   - dims gives N, T, E, R and cap_rows of the batch; H, x_dtype are not
 *     used, y_dtype where stated.  K and F are the product's own sizes:
 *     8 <= K, F <= 2^24, multiples of 8 (128 where stated).  N*cap stays below
 *     2^31 - 65536.
 *   - expert_offsets i32 [E+1] is moe_dispatch_count's output.  The rows of
 *     expert e on rank d = e / (E/N) are p = d*cap + (expert_offsets[e] -
 *     expert_offsets[d*E/N]) and the expert_counts[e] - 1 rows behind it, as
 *     far as they lie in the rank's region (rows over capacity were
 *     dropped).  Only these rows of the outputs are written; what other
 *     rows of the inputs hold (NaN, say) has no influence.
 *     Other contents lead to no access outside the arrays; for the products,
 *     offsets that descend or span more than N*T*R rows stand for no rows.
 *   - Outputs must not overlap inputs or each other (MOE_ERR_INVALID_ARG).
 *   - Array bases that a call reads by blocks must be 16-byte aligned (all
 *     but expert_offsets and the scales, which need 4).
 *   - Sums are f32; a result is rounded once, to nearest even.  Within a
 *     part of a sum the tensor core cuts off below the last place instead of
 *     rounding, about 1e-9 of the sum for each term, 5e-9 where all terms have
 *     one sign.  A part has 512 terms (f32 results: 5e-7 off at any length),
 *     2048 (bf16 results, sums that can be longer than 16384) or all of them
 *     (shorter ones: 8e-5 at most); parts are added up rounding to nearest.
 *     Results do not depend on scheduling: the same call gives the same bits.
 *   - The kernels need sm_103a's tensor memory: a block holds all 512
 *     columns of its SM.  A wait inside a kernel is bounded; one that gives
 *     up is reported by moe_take_device_error.
 * With N = E = R = 1 (expert_offsets = {0, T}, cap_rows = T) they are the
 * plain products of a shared expert or a dense layer.
 */
#ifndef MOE_EXPERT_H
#define MOE_EXPERT_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- what becomes of the sums ------------------------------------------- */
#define MOE_EXPERT_LINEAR 0 /* they are the result */
#define MOE_EXPERT_SWIGLU 1 /* h = g / (1 + exp(-g)) * u of the gate's and the up projection's sums g, u */

/* Product of each expert's rows with its matrix, in bf16.
 *   act MOE_EXPERT_LINEAR: y[p][f] = sum_k x[p][k] w[e][f][k]
 *     x   bf16 [N*cap][K], w bf16 [E][F][K]
 *     y   [N*cap][F] of dims->y_dtype; pre must be NULL
 *   act MOE_EXPERT_SWIGLU: g[p][f] = sum_k x[p][k] w[e][f][k],
 *     u[p][f] = sum_k x[p][k] w[e][F+f][k], y = silu(g) * u in f32
 *     x   bf16 [N*cap][K], w bf16 [E][2F][K] (gate rows, then up rows)
 *     y   bf16 [N*cap][F] whatever dims->y_dtype
 *     pre bf16 [N*cap][2F] or NULL (out): g and u rounded to bf16, for
 *         moe_expert_swiglu_grad (y comes from the unrounded sums). */
int moe_expert_gemm(const MoeDims *dims, int K, int F, int act, const void *x, const void *w,
                    const int32_t *expert_offsets, void *y, void *pre, void *stream);

/* Gradient of the linear product with respect to the rows:
 * dx[p][k] = sum_f dy[p][f] w[e][f][k].  dy bf16 [N*cap][F], w bf16 [E][F][K],
 * dx bf16 [N*cap][K].  (For the gated product pass 2F for F and
 * moe_expert_swiglu_grad's output for dy.) */
int moe_expert_gemm_dgrad(const MoeDims *dims, int K, int F, const void *dy, const void *w,
                          const int32_t *expert_offsets, void *dx, void *stream);

/* Gradient of the linear product with respect to the matrices:
 * dw[e][f][k] = sum over e's rows p of dy[p][f] x[p][k], 0 for an expert
 * without rows.  dy bf16 [N*cap][F], x bf16 [N*cap][K], dw [E][F][K] of
 * dw_dtype (MOE_BF16 or MOE_F32): written whole, not added to. */
int moe_expert_gemm_wgrad(const MoeDims *dims, int K, int F, const void *dy, const void *x,
                          const int32_t *expert_offsets, void *dw, int dw_dtype, void *stream);

/* Gradient of the gated activation: with s = 1 / (1 + exp(-g)),
 * dg = dh u s (1 + g (1 - s)), du = dh g s.
 *   pre  bf16 [N*cap][2F] (g, then u), dh bf16 [N*cap][F],
 *   dpre bf16 [N*cap][2F] (out): dg, then du. */
int moe_expert_swiglu_grad(const MoeDims *dims, int F, const void *pre, const void *dh,
                           const int32_t *expert_offsets, void *dpre, void *stream);

/* Product of each expert's rows with its matrix, both in e4m3 with block
 * scales; K % 128 == 0.
 *   xq       e4m3 [N*cap][K], x_scales f32 [N*cap][K/128]: as
 *            moe_dispatch_pack_quant or moe_dispatch_fused_quant write them
 *   wq       e4m3 [E][W][K], w_scales f32 [E][ceil(W/128)][K/128]: one scale
 *            per 128 x 128 block; W = F (linear) or 2F (gated: gate rows,
 *            then up rows)
 *   sum      s[p][f] = sum_b x_scales[p][b] w_scales[e][f/128][b]
 *            (sum over k in block b of xq[p][k] wq[e][f][k]), every sum in f32
 *   act MOE_EXPERT_LINEAR: y [N*cap][F] of dims->y_dtype, y_scales NULL
 *   act MOE_EXPERT_SWIGLU (F % 128 == 0): h = silu(g) * u in f32, then
 *            quantised: per 128 features of a row scale = fl32(amax/448) and code =
 *            e4m3 of h * fl32(1/scale), to nearest even, saturated (amax = 0:
 *            scale 0, codes 0): y e4m3 [N*cap][F] and y_scales f32
 *            [N*cap][F/128], the layout moe_dispatch_pack_quant writes, ready
 *            to be the next product's rows.  Infinite or NaN sums give
 *            unspecified codes.
 * Backward passes use the bf16 calls: the fp8 dispatch is a serving form. */
int moe_expert_gemm_fp8(const MoeDims *dims, int K, int F, int act, const void *xq, const float *x_scales,
                        const void *wq, const float *w_scales, const int32_t *expert_offsets, void *y,
                        float *y_scales, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERT_H */
