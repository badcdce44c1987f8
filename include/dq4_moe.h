/*
 * dq4_moe.h -- C ABI of a mixture-of-experts layer for a few tokens: the router,
 * and the chosen experts' gated feed-forward blocks over nested 4-bit weights.
 *
 *     router   l_e = sum_k x_k r_ek + bias_e             (64-bit sums of exact products)
 *              ids = the top_k experts of largest l, ties to the lower index
 *              weights = exp(l_id) / sum of exp(l) over the chosen experts
 *                        (renormalize != 0) or over all of them      (FP32)
 *     experts  h_te = T(act(x_t Wg_e^T) * (x_t Wu_e^T))
 *              y_t = T(sum_j weights_tj (h_te Wd_e^T) + residual_t), e = ids_tj
 *
 * T is the call's 16-bit type (DQ4_F16 or DQ4_BF16).  The experts' matrices are
 * stacked by rows: gate and up are nested 4-bit weights (dq4_weight_t of
 * dq4_linear.h) of (n_experts n_ff) x n_in elements, down one of (n_experts
 * n_in) x n_ff.  Their elements enter the products as exactly the values
 * dq4_nested_dequant writes for T; products are summed in FP32, h and y are
 * rounded once.  h is an operand of the down product and has T's range: in FP16
 * an h beyond 65504 is an infinity, as it is in dq4_gated_fused's output, and its
 * token's y infinities and NaN.
 *
 * Matrices are row-major with unit stride along a row and the row stride (in
 * elements) given as ld_*; a single row's stride is not looked at.  Only the m
 * rows and their columns are read or written.  No pointer but the workspace's
 * has to be aligned beyond its element type; 4-byte aligned packed codes and
 * row lengths that are multiples of 32 take the fastest path, multiples of 8
 * the next.  `residual` may be `y` itself (same pointer and row stride); no
 * other output may overlap an input, a weight or another output, and the
 * workspace none of them.  (Nothing is refused for it here; the Python binding
 * does.)
 *
 * workspace: caller-owned device memory, 256-byte aligned, of at least the
 * bytes that the call's *_workspace_bytes function returns.  Its contents do
 * not matter before the call, and after it the workspace holds nothing of use.
 * Calls that may overlap in time must not share one.
 *
 * Ownership, ordering and errors are as in dq4.h: everything is enqueued on
 * `stream` and can be captured into a graph, nothing is allocated, kept or
 * synchronized; arguments are checked before anything is enqueued.  Results
 * are deterministic for a given device, shape, and alignment of x and the
 * packed codes; for another number of tokens the sums may run in another order.
 *   DQ4_EINVAL       negative size, row stride below the row length, missing
 *                    pointer, unknown type or activation, top_k below 1, or
 *                    above n_experts (dq4_moe_route alone), workspace too small
 *                    or not 256-byte aligned
 *   DQ4_EUNSUPPORTED n_experts above 512, top_k above 16, more than 64 tokens
 *                    (dq4_moe_fused; 2^21 for the router), n_ff or n_in above
 *                    2^17, n_experts n_ff n_in above 2^40, block layout that
 *                    dq4_nested_dequant rejects, gate and up with different
 *                    block sizes
 *   DQ4_EHIP         a launch failed
 */
#ifndef DQ4_MOE_H
#define DQ4_MOE_H

#include "dq4.h"
#include "dq4_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DQ4_MOE_MAX_TOKENS 64
#define DQ4_MOE_MAX_EXPERTS 512
#define DQ4_MOE_MAX_TOP_K 16

/*
 * x: m x n_in, T.  router: n_experts x n_in, T, dense.  bias: n_experts FP32
 * values, or NULL.  ids: m x top_k, weights: m x top_k, dense, in order of
 * falling logits.
 * A bias of minus infinity masks its expert, whose logit is then minus infinity
 * whatever its row of the router and the token hold.  An expert whose logit is
 * minus infinity is not chosen; places that no expert is left for get id -1 and
 * weight 0.  A NaN logit ranks below every number; a token with one, or with a
 * logit of plus infinity, gets NaN for its weights.
 */
dq4_status_t dq4_moe_route(const void *x, int64_t m, int64_t n_in, int64_t ld_x, int32_t dtype,
                           const void *router, const float *bias, int32_t n_experts, int32_t top_k,
                           int32_t renormalize, int32_t *ids, float *weights, void *workspace,
                           int64_t workspace_bytes, void *stream);

/* 0 for sizes the call rejects.  Host only. */
int64_t dq4_moe_route_workspace_bytes(int64_t m, int32_t n_experts);

/*
 * x: m x n_in.  ids, weights: m x top_k, dense, as dq4_moe_route writes them or
 * from any other router.  An id outside 0 .. n_experts - 1 stands for no expert
 * (a padded token has only those); one that occurs twice in a row counts with
 * the sum of its weights, and top_k may exceed n_experts.  activation: any but
 * DQ4_ACT_NONE.  residual: m x n_in, or NULL.  y: m x n_in.
 * m == 0 or n_in == 0 is a no-op; n_ff == 0 is an empty sum (down's codebooks are
 * asked for all the same).
 */
dq4_status_t dq4_moe_fused(const dq4_weight_t *gate, const dq4_weight_t *up,
                           const dq4_weight_t *down, int32_t n_experts, int64_t n_ff, int64_t n_in,
                           int32_t dtype, int32_t activation, const void *x, int64_t m, int64_t ld_x,
                           const int32_t *ids, const float *weights, int32_t top_k,
                           const void *residual, int64_t ld_residual, void *y, int64_t ld_y,
                           void *workspace, int64_t workspace_bytes, void *stream);

/* 0 for sizes the call rejects.  Host only. */
int64_t dq4_moe_fused_workspace_bytes(int32_t n_experts, int64_t n_ff, int64_t n_in, int64_t m,
                                      int32_t top_k);

#ifdef __cplusplus
}
#endif

#endif /* DQ4_MOE_H */
