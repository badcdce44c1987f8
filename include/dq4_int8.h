/*
 * dq4_int8.h -- C ABI of the LLM.int8 linear layer: tokens quantized to 8-bit
 * codes, the product of 8-bit codes with a scale for each token and each
 * output channel, and its gradient.
 *
 * The weight of every call is what dq4_int8_prep takes: n_out x n_in codes CB
 * (row-major, dense) and one FP32 scale SCB[n] per row, the row's largest
 * magnitude, so that an element stands for CB SCB / 127.  T is the call's
 * 16-bit type (DQ4_F16 or DQ4_BF16).
 *
 *     quantization  s_i = max |x_ij| over the elements below the threshold,
 *                   codes_ij = round(127 x_ij / s_i), half to even, exactly
 *     product       y = T(sum_j codes_ij CB_nj s_i SCB_n / 127^2
 *                         + sum_l x[i][c_l] W[n][c_l] + bias_n + residual_in)
 *     backward      dx = T(dy W),  dbias = sum over rows of dy       (FP32)
 *     W             T(fl32(fl32(CB SCB) R127)), R127 the FP32 value nearest
 *                   1/127: the elements that dq4_int8_prep writes
 *
 * The sum over j is exact, in 32-bit integers, and scales may have any size: no
 * step leaves FP32's range where its value does not.  The other sums are FP32, and
 * every output is rounded once.  Columns c_l are the outliers, those in which
 * some element's magnitude reaches the threshold: their codes are 0, and they
 * enter in 16 bits.  Their list stays on the device, as the quantization
 * leaves it: outliers[0] is their number, outliers[1 ..] the columns in
 * ascending order, then -1; 1 + n_in values in all.
 *
 * Matrices are row-major with unit stride along a row and the row stride (in
 * elements) given as ld_*; a single row's stride is not looked at.  Only the m
 * rows and their columns are read or written.  No pointer but the workspace's
 * has to be aligned beyond its element type; 16-byte aligned rows take the
 * fastest paths.  `residual` may be `y` itself (same pointer and row stride);
 * no other output may overlap an input or another output, and the workspace
 * none of them.  (Nothing is refused for it here; the Python binding does.)
 *
 * workspace: caller-owned device memory, 256-byte aligned, of at least the
 * bytes that the call's *_workspace_bytes function returns.  Its contents do
 * not matter before the call, and after it the workspace holds nothing of use.
 * Calls that may overlap in time must not share one.
 *
 * Ownership, ordering and errors are as in dq4.h: everything is enqueued on
 * `stream` and can be captured into a graph, nothing is allocated, kept or
 * synchronized; arguments are checked before anything is enqueued.  Results
 * are deterministic for a given device and shape.
 *   DQ4_EINVAL       negative size, row stride below the row length, missing
 *                    pointer, unknown type, negative or NaN threshold,
 *                    workspace too small or not 256-byte aligned
 *   DQ4_EUNSUPPORTED n_in above 131071 (where a sum of products of 8-bit codes
 *                    could leave 32 bits; the backward call allows 2^21), m or
 *                    n_out above 2^21, a matrix of more than 2^38 elements
 *   DQ4_EHIP         a launch failed
 */
#ifndef DQ4_INT8_H
#define DQ4_INT8_H

#include "dq4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * codes (m x n_in) and scales (m) of the rows of x (m x n_in, T).
 *
 * threshold > 0: the columns that hold an element with a magnitude not below
 * it, infinities and NaN included, are the outliers: listed in `outliers`
 * (1 + n_in values, all of them written), their codes 0.  A row's scale is its
 * largest magnitude below the threshold, whatever its column.
 * threshold == 0: no column is, and `outliers` must be NULL.  The scale of a row
 * with an infinity or a NaN is NaN and its codes are 0, so that the product's
 * row is NaN.
 * A row without a magnitude above 0 has scale 0 and codes 0.
 */
dq4_status_t dq4_int8_quant(const void *x, int64_t m, int64_t n_in, int64_t ld_x, int32_t dtype,
                            float threshold, int8_t *codes, int64_t ld_codes, float *scales,
                            int32_t *outliers, void *workspace, int64_t workspace_bytes,
                            void *stream);

int64_t dq4_int8_quant_workspace_bytes(int64_t m, int64_t n_in, float threshold);

/*
 * The product.  codes: m x n_in, scales: m, as dq4_int8_quant writes them (any
 * codes from -128 to 127).  bias: n_out values of T, or NULL.  residual: m x
 * n_out of T, or NULL.  y: m x n_out.
 * x (m x n_in, T) and outliers: both, or both NULL for no outliers.  Only x's
 * outlier columns are read.  A count outside 0 .. n_in is taken as the nearest
 * of both; a column index outside 0 .. n_in - 1 reads nothing and gives NaN.
 * m == 0 or n_out == 0 is a no-op; n_in == 0 is an empty sum.
 */
dq4_status_t dq4_int8_linear(const int8_t *codes, int64_t m, int64_t ld_codes, const float *scales,
                             const int8_t *CB, const float *SCB, int64_t n_out, int64_t n_in,
                             int32_t dtype, const void *x, int64_t ld_x, const int32_t *outliers,
                             const void *bias, const void *residual, int64_t ld_residual, void *y,
                             int64_t ld_y, void *workspace, int64_t workspace_bytes, void *stream);

/* outliers: whether the call has some; of codes and CB the alignment matters. */
int64_t dq4_int8_linear_workspace_bytes(const int8_t *codes, int64_t m, int64_t ld_codes,
                                        const int8_t *CB, int64_t n_out, int64_t n_in,
                                        int32_t outliers);

/*
 * dy: m x n_out, T.  dx: m x n_in, T.  dbias: n_out FP32 values, overwritten
 * (m == 0 writes zeros), or NULL.  The weight is frozen.
 */
dq4_status_t dq4_int8_linear_backward(const int8_t *CB, const float *SCB, int64_t n_out,
                                      int64_t n_in, int32_t dtype, const void *dy, int64_t m,
                                      int64_t ld_dy, void *dx, int64_t ld_dx, float *dbias,
                                      void *workspace, int64_t workspace_bytes, void *stream);

int64_t dq4_int8_linear_backward_workspace_bytes(int64_t n_out, int64_t n_in, int64_t m,
                                                 const void *dy, int64_t ld_dy);

#ifdef __cplusplus
}
#endif

#endif /* DQ4_INT8_H */
