/*
 * int4vh_linear.h -- C ABI of the linear layer on packed int4 weights (same
 * library, libint4vh.so; status codes and error text as in int4vh.h).
 *
 * The weights are those of the output head's format (int4vh_requant.h packs
 * them): two values per byte, [N, K/2], in [-7, 7], one scale per input
 * channel.  The activations are 8-bit rows (int4vh_norm.h), into which the
 * channel scales have been folded:
 *
 *   acc[m, n] = sum_k codes[m, k] * q[n, k]                        (exact integer)
 *   y         = f32(acc[m, n]) * row_scales[m]
 *   y         = y * out_scales[n]                                  (optional)
 *   y         = y + f32(bias[n])                                   (optional)
 *   y         = activation(y):  none | max(y, 0) | y / 2 * erfc(-y / sqrt(2)) | y / (1 + exp(-y))
 *   out[m, n] = y + f32(residual[m, n])  (optional), rounded once to `dtype`
 *
 * Numerics.  The products run on the int8 matrix cores and their sums are
 * exact in 32 bits, so the results do not depend on the launch shape, on M or
 * on how the sum over k is split: a row gives the same bits alone and in a
 * batch.  The epilogue is binary32 in the order written, without fused
 * multiply-adds; the gelu as a whole has a relative error below (1.5 y^2 + 14)
 * 2^-24, in its lower tail too (where exp(-y^2 / 2) is subnormal, an error below
 * (|y| + 1) 2^-150 more), and the silu is -0 where exp(-y) overflows (y below
 * -88.7).  A row_scale that is NaN makes its row NaN; an infinite one
 * makes products infinite, and NaN where acc is 0, before the bias and the
 * activation.
 *
 * Layout (device memory owned by the caller): codes int8 [M, K], rows
 * codes_stride elements apart, 16-byte aligned rows; row_scales float32 [M];
 * packed_w uint8 [N, K/2], 16-byte aligned; out_scales float32 [N]; bias [N],
 * residual [M, N] and out [M, N] of `dtype` (INT4VH_ROWS_*), rows
 * residual_stride / out_stride elements apart, aligned to their element.  out
 * may be residual itself with the same stride, and may overlap nothing else.
 * Weights outside [-7, 7] (nibble 0x8, which stands for -8) are computed
 * with as such.
 *
 * Workspace.  Calls of some shapes split the sum over k and need
 * linear_int4_rows_workspace_bytes(M, N, K) bytes (0 for the others), 256-byte
 * aligned, no initialisation; its contents mean nothing between calls.  Two
 * calls in flight at the same time must not share it.
 *
 * Calls are asynchronous on `stream`, allocate nothing and may be captured in
 * a graph.
 *
 * Errors (host validation before any launch): INT4VH_EINVAL for M < 1, N < 1,
 * K < 32 or K % 32 != 0, an unknown activation or dtype, a required pointer
 * that is NULL, a stride below the row's length (M > 1);
 * INT4VH_EALIGN for a misaligned pointer or a codes_stride that is no multiple
 * of 16 (M > 1); INT4VH_EWORKSPACE for a workspace that is too small;
 * INT4VH_EUNSUPPORTED for K > 65536, N > 2^24, M > 2^20, M * N >= 2^40 or a
 * codes_stride of 2^24 or more (M > 1); INT4VH_EHIP for a launch failure.
 */
#ifndef INT4VH_LINEAR_H
#define INT4VH_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#include "int4vh_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    INT4VH_ACT_NONE = 0,
    INT4VH_ACT_RELU = 1,
    INT4VH_ACT_GELU = 2,
    INT4VH_ACT_SILU = 3
};

/* Bytes of workspace a call of these sizes needs on the current device (0 if
 * it needs none or the sizes are invalid).  Launches nothing. */
size_t linear_int4_rows_workspace_bytes(int M, int N, int K);

int linear_int4_rows(const int8_t *codes, int64_t codes_stride, const float *row_scales, const uint8_t *packed_w,
                     const float *out_scales, const void *bias, int activation, const void *residual,
                     int64_t residual_stride, int M, int N, int K, void *out, int64_t out_stride, int dtype,
                     void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* INT4VH_LINEAR_H */
