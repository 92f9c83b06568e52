/*
 * moe_grad.h -- C ABI of the routing steps' gradients in libmoe_route.so:
 * what a training step needs of combine, dispatch and the router, next to the
 * gradients of the experts' products (moe_expert.h).
 *
 * "Efficient and portable mixture-of-experts communication", sections
 * "Dispatch" and "Combine": tokens are copied to their experts' rows and the
 * results come back weighted; here the same two moves in the other direction.
 *
 * The conventions of moe_route.h hold: device pointers owned by the caller,
 * dense row-major arrays, work enqueued on `stream`, no host
 * synchronisation, nothing allocated and no workspace, grids that do not
 * depend on routing, argument errors reported before anything is enqueued.
 * Results must not overlap the other arrays of a call (MOE_ERR_INVALID_ARG)
 * but where stated.  Sums are f32 or longer, taken in a fixed order: the same
 * call gives the same bits.
 *
 * A training step in order: moe_combine_grad, the gradients of the experts'
 * products, moe_dispatch_grad, moe_route_grad.
 */
#ifndef MOE_GRAD_H
#define MOE_GRAD_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Gradient of moe_combine, out[g] = sum_k topk_w[g][k] y[pos[g][k]]:
 *   dout    [N*T][H] of y_dtype (in): gradient of out
 *   y       [N*cap][H] of y_dtype (in), pos i32 [N*T][R], topk_w f32 [N*T][R]:
 *           what moe_combine read
 *   dy      [N*cap][H] of y_dtype (out): dy[pos[g][k]] = topk_w[g][k] dout[g],
 *           rounded once; other rows are left as they were
 *   dtopk_w f32 [N*T][R] (out): sum over h of dout[g][h] y[pos[g][k]][h]
 * Pairs with pos < 0 (or outside [0, N*cap)) have no row and get dtopk_w = 0.
 * Rows of two pairs, which moe_dispatch_count never gives, end up with one of
 * their products, not with the sum.
 * dout, y and dy must be 16-byte aligned. */
int moe_combine_grad(const MoeDims *dims, const void *dout, const void *y, const int32_t *pos,
                     const float *topk_w, void *dy, float *dtopk_w, void *stream);

/* Gradient of moe_dispatch_pack, packed_x[pos[g][k]] = x[g]:
 *   dpacked [N*cap][H] of x_dtype (in): gradient of the packed rows
 *   pos     i32 [N*T][R] (in)
 *   add     [N*T][H] of x_dtype or NULL (in): the tokens' gradient from
 *           elsewhere (a shared expert, the router's own product); may be dx,
 *           which is then added to
 *   dx      [N*T][H] of x_dtype (out): add[g] + sum_k dpacked[pos[g][k]], in
 *           f32 in this order, rounded once
 * Pairs with pos < 0 (or outside [0, N*cap)) contribute nothing.  x_dtype is
 * MOE_BF16 or MOE_F32 (the fp8 dispatch is a serving form). */
int moe_dispatch_grad(const MoeDims *dims, const void *dpacked, const int32_t *pos, const void *add, void *dx,
                      void *stream);

/* Gradient of moe_route_topk's weights with respect to the logits, the chosen
 * experts being fixed.
 *   logits, bias, score_fn, renormalize   as in moe_route_topk
 *   topk_idx, topk_w                      what it wrote
 *   dtopk_w f32 [N*T][R] (in): gradient of topk_w (moe_combine_grad)
 *   dlogits f32 [N*T][E] (out), written whole
 *   dbias   f32 [E] or NULL (out): sum over the tokens of dlogits, the gradient
 *           of a bias that is added to the logits; with MOE_BIAS_SELECT_ONLY
 *           the bias has none and dbias must be NULL
 * With z = fl32(logit + bias) (the logit with MOE_BIAS_SELECT_ONLY), h = dtopk_w,
 * w = topk_w, d = sum_k h_k w_k:
 *   softmax                dlogit_e = p_e (h_e - d), p = softmax(z) over all E,
 *                          h_e = 0 where e was not chosen
 *   softmax, renormalised  dlogit_e = w_k (h_k - d) for e = topk_idx[k], else 0
 *   sigmoid                dlogit_e = w_k h_k / (1 + exp(z_e)), else 0
 *   sigmoid, renormalised  dlogit_e = w_k (h_k - d) / (1 + exp(z_e)), else 0
 * Logits of -infinity have weight and gradient 0; softmax over a token's logits
 * that are all -infinity gives zeros, over any NaN among them NaN.  Weights
 * that are NaN (chosen scores that are all 0, renormalised) give NaN in their
 * token's row.  An expert that a token names twice gets both parts; ids
 * outside [0, E) take no part. */
int moe_route_grad(const MoeDims *dims, const float *logits, const float *bias, int score_fn, int renormalize,
                   const int32_t *topk_idx, const float *topk_w, const float *dtopk_w, float *dlogits,
                   float *dbias, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GRAD_H */
