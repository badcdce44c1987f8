/*
 * dq4_linear.h -- C ABI of the fused products over nested 4-bit weights: the
 * linear layer with bias, activation and residual in its epilogue, the gated
 * half of a feed-forward block, and the backward pass of each.
 *
 * The weight of every call is the frozen nested 4-bit weight of dq4.h.  Its
 * elements enter the products as exactly the values dq4_nested_dequant writes
 * for the call's 16-bit type T (DQ4_F16 or DQ4_BF16), for every number of
 * rows m; products are summed in FP32 and every result is rounded to T once.
 * The backward products take dz, dgate and dup as rounded to T.
 *
 *     linear            z = x W^T + bias
 *                       pre = T(z),  y = T(act(z) + residual)
 *     linear backward   dz = T(dy * act'(pre)),  dx = T(dz W),
 *                       dbias = sum over rows of dy * act'(pre)    (FP32)
 *     gated             g = x Wg^T,  u = x Wu^T
 *                       gate_pre = T(g),  up_pre = T(u),  h = T(act(g) * u)
 *     gated backward    dgate = T(dh * up_pre * act'(gate_pre)),
 *                       dup = T(dh * act(gate_pre)),
 *                       dx = T(dgate Wg + dup Wu)                  (one FP32 sum)
 *
 * act and act' are evaluated in FP32 on the FP32 pre-activation (forward) or
 * on the saved one (backward).  A low-rank (LoRA) term enters as `residual`
 * of a call without activation; its gradients take dz, dgate and dup.
 * A NaN pre-activation gives NaN with every activation, forward and backward.
 * At a saved pre-activation of plus or minus infinity, which FP16 reaches by
 * overflow, the backward calls take act' as 1 or 0 and act as infinity or 0,
 * their limits.
 *
 * Matrices are row-major with unit stride along a row and the row stride
 * (in elements) given as ld_*; a single row's stride is not looked at.  Only
 * the m rows and their columns are read or written: what lies between the
 * rows of a strided matrix, and behind the last row, stays as it was.
 * No pointer but the workspace's has to be aligned beyond its element type;
 * 16-byte aligned rows and 4-byte aligned packed codes take the fastest paths.
 * `residual` may be `y` itself (same pointer and row stride); no other output
 * may overlap an input, a weight or another output, and the workspace none of
 * them.  (Nothing is refused for it here; the Python binding does.)
 *
 * workspace: caller-owned device memory, 256-byte aligned, of at least the
 * bytes that the call's *_workspace_bytes function returns with `least` = 1;
 * with the bytes of `least` = 0 a decoded weight fits whole, with fewer it
 * passes through in windows of output columns.  Its contents do not matter
 * before the call, and after it the workspace holds nothing of use.  Calls
 * that may overlap in time must not share one.  A workspace changes speed
 * only, never results.
 *
 * Ownership, ordering and errors are as in dq4.h: everything is enqueued on
 * `stream` and can be captured into a graph, nothing is allocated, kept or
 * synchronized; arguments are checked before anything is enqueued.
 * Results are deterministic for a given device, shape, and alignment of the
 * packed codes; for another number of rows the sums may run in another order.
 *   DQ4_EINVAL       negative size, row stride below the row length, missing
 *                    pointer, unknown type or activation, workspace too small
 *                    or not 256-byte aligned
 *   DQ4_EUNSUPPORTED block layout that dq4_nested_dequant rejects, two
 *                    weights with different block sizes, m, n_out or n_in
 *                    above 2^21, m n_out or m n_in above 2^39
 *   DQ4_EHIP         a launch failed
 */
#ifndef DQ4_LINEAR_H
#define DQ4_LINEAR_H

#include "dq4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A nested 4-bit weight of n_out x n_in elements, row-major: the first six
 * arguments and the two block sizes of dq4_nested_dequant. */
typedef struct dq4_weight {
    const uint8_t *packed;
    const uint8_t *scale_codes;
    const float *nested_absmax;
    const float *scale_codebook;
    const float *codebook4;
    float offset;
    int32_t blocksize;
    int32_t nested_blocksize;
} dq4_weight_t;

enum {
    DQ4_ACT_NONE = 0,      /* z                          (linear calls only) */
    DQ4_ACT_RELU = 1,      /* max(z, 0); slope 0 at 0                        */
    DQ4_ACT_SILU = 2,      /* z / (1 + exp(-z))                              */
    DQ4_ACT_GELU = 3,      /* z/2 * erfc(-z / sqrt 2)                        */
    DQ4_ACT_GELU_TANH = 4  /* z/2 * (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
};

/*
 * y = T(act(x W^T + bias) + residual).
 * x: m x n_in.  bias: n_out values of T, or NULL.  residual: m x n_out of T,
 * or NULL.  y: m x n_out.  pre: m x n_out, the pre-activation z rounded to T
 * for the backward pass, or NULL.
 * m == 0 or n_out == 0 is a no-op; n_in == 0 is an empty sum.
 */
dq4_status_t dq4_linear_fused(const dq4_weight_t *w, int64_t n_out, int64_t n_in, int32_t dtype,
                              int32_t activation, const void *x, int64_t m, int64_t ld_x,
                              const void *bias, const void *residual, int64_t ld_residual,
                              void *y, int64_t ld_y, void *pre, int64_t ld_pre, void *workspace,
                              int64_t workspace_bytes, void *stream);

/* Workspace bytes of dq4_linear_fused for this weight and x (only the
 * alignment of w->packed, x and ld_x matters): the preferred size, or with
 * least != 0 the smallest the call accepts.  0 when the call needs none, and
 * for a missing weight or sizes the call rejects.  Host only. */
int64_t dq4_linear_fused_workspace_bytes(const dq4_weight_t *w, int64_t n_out, int64_t n_in,
                                         int64_t m, const void *x, int64_t ld_x, int32_t least);

/*
 * dz = T(dy * act'(pre)), dx = T(dz W), dbias = column sums of the unrounded
 * FP32 products dy * act'(pre).
 * dy: m x n_out.  pre: m x n_out, what the forward call saved; not read with
 * DQ4_ACT_NONE.  dz: m x n_out, written; with DQ4_ACT_NONE dz is dy, and the
 * argument must be NULL.  dx: m x n_in.  dbias: n_out FP32 values, overwritten
 * (m == 0 writes zeros), or NULL.
 */
dq4_status_t dq4_linear_fused_backward(const dq4_weight_t *w, int64_t n_out, int64_t n_in,
                                       int32_t dtype, int32_t activation, const void *dy,
                                       int64_t m, int64_t ld_dy, const void *pre, int64_t ld_pre,
                                       void *dx, int64_t ld_dx, void *dz, int64_t ld_dz,
                                       float *dbias, void *workspace, int64_t workspace_bytes,
                                       void *stream);

/* dz, ld_dz: of the matrix the product reads (dy with DQ4_ACT_NONE). */
int64_t dq4_linear_fused_backward_workspace_bytes(const dq4_weight_t *w, int64_t n_out,
                                                  int64_t n_in, int64_t m, const void *dz,
                                                  int64_t ld_dz, int32_t least);

/*
 * h = T(act(x Wg^T) * (x Wu^T)), both weights n_ff x n_in with one block size.
 * x: m x n_in.  h: m x n_ff.  gate_pre, up_pre: m x n_ff with one row stride
 * ld_pre, the two products rounded to T for the backward pass; both or
 * neither may be NULL.  activation: any but DQ4_ACT_NONE.
 */
dq4_status_t dq4_gated_fused(const dq4_weight_t *gate, const dq4_weight_t *up, int64_t n_ff,
                             int64_t n_in, int32_t dtype, int32_t activation, const void *x,
                             int64_t m, int64_t ld_x, void *h, int64_t ld_h, void *gate_pre,
                             void *up_pre, int64_t ld_pre, void *workspace,
                             int64_t workspace_bytes, void *stream);

int64_t dq4_gated_fused_workspace_bytes(const dq4_weight_t *gate, const dq4_weight_t *up,
                                        int64_t n_ff, int64_t n_in, int64_t m, const void *x,
                                        int64_t ld_x, int32_t least);

/*
 * dgate = T(dh * up_pre * act'(gate_pre)), dup = T(dh * act(gate_pre)),
 * dx = T(dgate Wg + dup Wu).
 * dh: m x n_ff.  gate_pre, up_pre: m x n_ff, row stride ld_pre.  dx: m x n_in.
 * dgate, dup: m x n_ff, row stride ld_dpre, written.
 */
dq4_status_t dq4_gated_fused_backward(const dq4_weight_t *gate, const dq4_weight_t *up,
                                      int64_t n_ff, int64_t n_in, int32_t dtype,
                                      int32_t activation, const void *dh, int64_t m,
                                      int64_t ld_dh, const void *gate_pre, const void *up_pre,
                                      int64_t ld_pre, void *dx, int64_t ld_dx, void *dgate,
                                      void *dup, int64_t ld_dpre, void *workspace,
                                      int64_t workspace_bytes, void *stream);

/* dgate, dup: of the matrices the product reads (their alignment matters). */
int64_t dq4_gated_fused_backward_workspace_bytes(const dq4_weight_t *gate,
                                                 const dq4_weight_t *up, int64_t n_ff,
                                                 int64_t n_in, int64_t m, const void *dgate,
                                                 const void *dup, int64_t ld_dpre,
                                                 int32_t least);

#ifdef __cplusplus
}
#endif

#endif /* DQ4_LINEAR_H */
