// linear_common.h -- what the linear layers share: waits and barriers, the
// epilogue's activations (not part of the C ABI).
#ifndef INT4VH_LINEAR_COMMON_H
#define INT4VH_LINEAR_COMMON_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "int4vh_linear.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace int4vh_detail {

constexpr int kWaitLgkm0 = 0xF | (0x3 << 14) | (0x7 << 4);

__device__ __forceinline__ void barrier_no_fence()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// LDS written and read by one wave alone: its accesses execute in order, so
// only the compiler has to be held back.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ float load_one(const void *p, size_t i, int dtype)
{
    return dtype == INT4VH_ROWS_F32 ? static_cast<const float *>(p)[i]
                                    : from_bits16(static_cast<const uint16_t *>(p)[i], dtype);
}

// y times the normal distribution function: y * q below 0 and y * (1 - q)
// above, where q = erfc(|y| / sqrt(2)) / 2 keeps its digits as it gets small
// (from 1 + erf nothing is left below -5.5).  q = exp(-y^2 / 2) * t P(t) with
// t = 1 / (1 + 0.2625 |y|); P is a least-squares fit of the scaled function,
// its weights moved towards the largest relative error until that was 0.34 u
// for |y| < 14.5 (u = 2^-24).  Relative error of the result: 3 u of the
// exponent y^2 / 2, and below 14 u of the polynomial, t, exp2 and the products:
// (1.5 y^2 + 14) u; measured 8 u down to -3 and 27 u down to -6.  4096 x 16384
// x 512 takes 100 us (111 with erff and its cancellation, 127 with erfcf).
__device__ __forceinline__ float gelu(float y)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.2625f, fabsf(y), 1.0f));
    float p = 0.03052651f;
    p = __builtin_fmaf(p, t, -0.14775364f);
    p = __builtin_fmaf(p, t, 0.23259342f);
    p = __builtin_fmaf(p, t, -0.13092719f);
    p = __builtin_fmaf(p, t, 0.14744487f);
    p = __builtin_fmaf(p, t, 0.056568123f);
    p = __builtin_fmaf(p, t, 0.10263485f);
    p = __builtin_fmaf(p, t, 0.10416468f);
    p = __builtin_fmaf(p, t, 0.10474835f);
    const float q = p * t * exp2f(y * y * -0.72134752f);
    return y * (y < 0.0f ? q : 1.0f - q);
}

// One uniform branch for kN values.
template <int kN>
__device__ __forceinline__ void activate(float (&y)[kN], int activation)
{
    if (activation == INT4VH_ACT_RELU) {
#pragma unroll
        for (int r = 0; r < kN; ++r)
            y[r] = y[r] < 0.0f ? 0.0f : y[r];      // a NaN stays one
    } else if (activation == INT4VH_ACT_GELU) {
#pragma unroll
        for (int r = 0; r < kN; ++r)
            y[r] = gelu(y[r]);
    } else if (activation == INT4VH_ACT_SILU) {
#pragma unroll
        for (int r = 0; r < kN; ++r)
            y[r] = y[r] / (1.0f + expf(-y[r]));
    }
}

} // namespace int4vh_detail

#endif // INT4VH_LINEAR_COMMON_H
