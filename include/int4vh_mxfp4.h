/*
 * int4vh_mxfp4.h -- C ABI of rows in microscaled 4-bit floating point (MXFP4)
 * and of the linear layer between two matrices in that format (same library,
 * libint4vh.so; status codes and error text as in int4vh.h).
 *
 * The format: 32 consecutive channels share a scale 2^(s - 127), s one byte
 * (255: the 32 values are NaN); a value is 4 bits, sign, two bits of exponent
 * and one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4 or 6.  A byte holds two, the even
 * channel in the low half.  A matrix [M, K] is codes uint8 [M, K/2] and scales
 * uint8 [M, K/32].
 *
 * quantize_rows_mxfp4, for each 32 channels x of a row:
 *   peak = max |x|;  s = clamp(floor(log2(peak)) - 2 + 127, 0, 254), 0 for peak 0
 *   code = x / 2^(s - 127), rounded to the nearest value (ties to the even code),
 *          6 beyond 6 (at most a quarter of the value is lost); the sign stays
 *   a NaN or an infinity among them: s = 255, codes 0
 * dequantize_rows_mxfp4: the values, rounded once to `dtype` (exact in binary32
 * but for what overflows it).
 *
 * linear_mxfp4_rows, x the rows and w the weights that the codes stand for:
 *   y         = sum_k x[m, k] * w[n, k]
 *   y         = y + f32(bias[n])                                   (optional)
 *   y         = activation(y), as in int4vh_linear.h
 *   out[m, n] = y + f32(residual[m, n])  (optional), rounded once to `dtype`
 *
 * Numerics.  The products run on the scaled 4-bit matrix cores: products are
 * exact, sums are binary32.  Their order depends on M, N, K and the device alone:
 * the same call gives the same bits, another number of rows may not.
 * The epilogue is binary32 in the order written, without fused multiply-adds.
 *
 * Layout (device memory owned by the caller): x [M, H] of `dtype`, rows x_stride
 * elements apart, aligned to its element.  codes, scales: contiguous; codes of
 * the linear layer and of dequantize 16-byte aligned, the quantisation's 4-byte
 * aligned.  bias [N], residual [M, N] and out [M, N] of `dtype`, rows
 * residual_stride / out_stride elements apart, aligned to their element.  out may
 * be residual itself with the same stride, and may overlap nothing else.
 *
 * Workspace.  Calls of some shapes split the sum over k and need
 * linear_mxfp4_rows_workspace_bytes(M, N, K) bytes (0 for the others), 256-byte
 * aligned, no initialisation; its contents mean nothing between calls.  Two
 * calls in flight at the same time must not share it.
 *
 * Calls are asynchronous on `stream`, allocate nothing and may be captured in
 * a graph.
 *
 * Errors (host validation before any launch): INT4VH_EINVAL for M < 1, N < 1, H
 * or K below 32 or no multiple of 32, an unknown activation or dtype, a required
 * pointer that is NULL, a stride below the row's length (M > 1); INT4VH_EALIGN
 * for a misaligned pointer; INT4VH_EWORKSPACE for a workspace that is too small;
 * INT4VH_EUNSUPPORTED for H or K > 65536, N > 2^24, M > 2^20 (the linear layer)
 * or M * N >= 2^40; INT4VH_EHIP for a launch failure.
 */
#ifndef INT4VH_MXFP4_H
#define INT4VH_MXFP4_H

#include <stddef.h>
#include <stdint.h>

#include "int4vh_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

int quantize_rows_mxfp4(const void *x, int64_t x_stride, int dtype, int M, int H, uint8_t *codes, uint8_t *scales,
                        void *stream);

int dequantize_rows_mxfp4(const uint8_t *codes, const uint8_t *scales, int M, int H, void *out, int dtype,
                          void *stream);

/* Bytes of workspace a call of these sizes needs on the current device (0 if
 * it needs none or the sizes are invalid).  Launches nothing. */
size_t linear_mxfp4_rows_workspace_bytes(int M, int N, int K);

int linear_mxfp4_rows(const uint8_t *codes, const uint8_t *scales, const uint8_t *w_codes, const uint8_t *w_scales,
                      const void *bias, int activation, const void *residual, int64_t residual_stride, int M, int N,
                      int K, void *out, int64_t out_stride, int dtype, void *workspace, size_t workspace_bytes,
                      void *stream);

#ifdef __cplusplus
}
#endif

#endif /* INT4VH_MXFP4_H */
