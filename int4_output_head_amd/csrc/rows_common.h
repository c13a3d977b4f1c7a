// rows_common.h -- element types shared by the row operators (not part of the
// C ABI).
#ifndef INT4VH_ROWS_COMMON_H
#define INT4VH_ROWS_COMMON_H

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "int4vh_norm.h"

namespace int4vh_detail {

// 16 / 8 bytes at the alignment of their elements (the hardware takes
// unaligned vector accesses)
struct __attribute__((packed, aligned(2))) Words2 { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) Words4 { uint32_t w[4]; };
struct __attribute__((packed, aligned(1))) Pair1 { uint32_t w[2]; };
struct __attribute__((packed, aligned(2))) Pair2 { uint32_t w[2]; };

__device__ __forceinline__ float from_bits16(uint32_t b, int dtype)
{
    return dtype == INT4VH_ROWS_F16 ? __half2float(__ushort_as_half((unsigned short)b)) : __uint_as_float(b << 16);
}

// binary32 -> bfloat16 bits, round to nearest even (one instruction here); a
// NaN stays one
__device__ __forceinline__ uint32_t to_bf16(float f)
{
    return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

__device__ __forceinline__ uint32_t to_bits16(float f, int dtype)
{
    return dtype == INT4VH_ROWS_F16 ? (uint32_t)__half_as_ushort(__float2half_rn(f)) : to_bf16(f);
}

inline bool rows_aligned(const void *p, size_t al)
{
    return ((uintptr_t)p % al) == 0;
}

inline bool rows_known(int dtype)
{
    return dtype == INT4VH_ROWS_F16 || dtype == INT4VH_ROWS_BF16 || dtype == INT4VH_ROWS_F32;
}

inline size_t rows_size(int dtype)
{
    return dtype == INT4VH_ROWS_F32 ? 4 : 2;
}

} // namespace int4vh_detail

#endif // INT4VH_ROWS_COMMON_H
