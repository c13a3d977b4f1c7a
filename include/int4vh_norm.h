/*
 * int4vh_norm.h -- C ABI of the row operators in front of the int4 products
 * (same library, libint4vh.so; status codes and error text as in int4vh.h).
 *
 * The hidden states that the verify calls take are the output of the model's
 * final residual addition and root-mean-square norm; the 8-bit activations of
 * linear_int4_rows (int4vh_linear.h) are the output of a norm, or of any other
 * layer, rounded to 8 bits with one scale per row.  For each of M rows:
 *
 *   h[i]     = f32(x[i]) + f32(residual[i])        (h = f32(x) without a residual)
 *   sum[i]   = h[i], rounded to the rows' type      (the residual stream; optional)
 *   rstd     = 1 / sqrt(sum_i h[i]^2 / H + eps)
 *   rms_norm_rows:       out[i] = (h[i] * rstd) * f32(weight[i]), rounded to out_dtype
 *   rms_norm_rows_int8:  t[i] = (h[i] * f32(weight[i])) * f32(channel_scales[i])
 *                        peak = max_i |t[i]|
 *                        codes[i] = rint(t[i] * (127 / peak))       in [-127, 127]
 *                        row_scale = (peak * rstd) / 127
 *                        so that codes[i] * row_scale is the normed row
 *                        (times the channel scale) to within half a step
 *   quantize_rows_int8:  the same with rstd = 1 and weight = 1 (no norm)
 *
 * channel_scales (binary16 [H], NULL for none) are the per-channel scales of a
 * packed int4 matrix (int4vh_requant.h): folded into the activations here, as
 * the verify calls do, they leave the weights pure integers.
 *
 * Numerics.  Everything is binary32, one rounding per operation in the order
 * written (the sum of squares in an order that depends on H alone: a row gives
 * the same bits in every batch).
 * The norm uses h before it is rounded to the rows' type.  The codes do not
 * depend on rstd.  A NaN or an infinity in a row makes that row's outputs NaN
 * or infinite as the formulas do; in 8 bits its codes are 0 and its row_scale
 * is NaN or infinite.  A row whose peak is below 2^-100 has codes 0 and
 * row_scale 0.  Rows of any finite size are normed as the formulas say: where
 * mean h^2 + eps overflows or is below 2^-80, the squares are summed at a scale
 * of another power of two, which rounds nothing.
 *
 * Layout.  x and residual: [M, H] of `dtype`, rows x_stride / residual_stride
 * elements apart (at least H, or any value when M == 1), channels contiguous.
 * sum_out: [M, H] of `dtype`, contiguous, NULL to skip; it may be x or
 * residual itself where those are contiguous.  weight: [H] of weight_dtype.
 * out: [M, H] of out_dtype; codes: int8 [M, H]; row_scales: float32 [M];
 * contiguous.  No output may overlap another buffer otherwise.  Rows need no
 * alignment beyond their element's.
 *
 * Calls are asynchronous on `stream`, allocate nothing, use no workspace and
 * may be captured in a graph; calls on different streams are independent.
 *
 * Errors (host validation before any launch): INT4VH_EINVAL for M < 1, H < 1,
 * an unknown dtype, a stride below H (M > 1), eps negative or not finite, a
 * required pointer that is NULL, or a sum_out without a residual;
 * INT4VH_EALIGN for a pointer that is not aligned to its element;
 * INT4VH_EUNSUPPORTED for H > 8192 (quantize_rows_int8: 65536, the linear
 * layers' limit); INT4VH_EHIP for a launch failure.
 */
#ifndef INT4VH_NORM_H
#define INT4VH_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "int4vh.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows, weights and outputs (the first two as in
 * int4vh_requant.h). */
enum {
    INT4VH_ROWS_F16 = 0,
    INT4VH_ROWS_BF16 = 1,
    INT4VH_ROWS_F32 = 2
};

int rms_norm_rows(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, int dtype,
                  const void *weight, int weight_dtype, int M, int H, float eps, void *sum_out, void *out,
                  int out_dtype, void *stream);

int rms_norm_rows_int8(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, int dtype,
                       const void *weight, int weight_dtype, const void *channel_scales, int M, int H, float eps,
                       void *sum_out, int8_t *codes, float *row_scales, void *stream);

int quantize_rows_int8(const void *x, int64_t x_stride, int dtype, const void *channel_scales, int M, int H,
                       int8_t *codes, float *row_scales, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* INT4VH_NORM_H */
