// norm.hip -- the row operators in front of the int4 products, for MI355X
// (gfx950): the residual addition with the root-mean-square norm that gives
// the verify calls their hidden states, and the same rows in 8 bits with one
// scale per row (formulas and order of rounding in int4vh_norm.h).
//
// Bound by HBM for many rows and by latency for few: x and the residual are
// read once, the sum and the normed row written once, and nothing else moves
// (weights stay in registers).  A row lives in the registers of one workgroup,
// 8 consecutive channels per thread, so one pass suffices: the sum of squares
// and the largest |t| of the row come out of one reduction, because t = (h *
// weight) * channel_scale does not depend on rstd -- the factor rstd is common
// to the row and goes into its scale alone.  Workgroups walk over rows with a
// stride of the grid and keep their channels' weights.  Rows whose squares
// leave binary32 are summed a second time at another scale.  (Two chunks of 8 per
// thread, half the waves: 47.3 us against 43.6 for 4096 x 8192 bfloat16 rows
// with residual, graph-timed, and 5.1 against 3.9 for one row in 8 bits.)
//
// Loads are 16 bytes wide whatever the rows' alignment (the hardware splits
// unaligned ones); only the thread that holds the last, partial chunk of a row
// goes element by element.
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>

#include "int4vh.h"
#include "int4vh_internal.h"
#include "int4vh_norm.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace {

using namespace int4vh_detail;

constexpr int kMaxThreads = 1024;
constexpr int kMaxLong = 65536;           // channels of a row in 8 bits without a norm
constexpr float kTinyPeak = 0x1p-100f;    // rows below it have no finite 127 / peak worth using
// Rows whose mean square + eps would overflow (from an rms of 2^57.5 on, for
// 8192 channels) or is below kLowMean, where squares get lost to subnormal
// numbers, are summed once more at another scale: kDown, at which squares
// reach 2^96 and their sum 2^109, or kUp, at which the smallest subnormal
// number squares to 2^-118 and a sum stays below 2^113.  Looking for them costs
// 0.1 us at 16 rows of 5120 bfloat16 channels (3.7 us) and 0.3 at 1021 (10.0).
constexpr float kLowMean = 0x1p-80f, kDown = 0x1p-80f, kUp = 0x1p90f;

struct NormArgs {
    const void *x;
    const void *residual;      // or null
    long long x_stride, residual_stride;
    const void *weight;        // [H] of weight_dtype, or null (quantize_rows_int8)
    const uint16_t *channel;   // binary16 [H], or null
    void *sum_out;             // or null
    void *out;                 // [M, H] of out_dtype (norm)
    int8_t *codes;             // [M, H] (8 bits)
    float *row_scales;         // [M]
    int M, H;
    int weight_dtype, out_dtype;
    float eps;
};

// Channels c .. c+7 of a row, as binary32.
template <int kDtype>
__device__ __forceinline__ void load8_whole(const void *row, int c, float (&v)[8])
{
    if constexpr (kDtype == INT4VH_ROWS_F32) {
        const Words4 a = *reinterpret_cast<const Words4 *>(static_cast<const float *>(row) + c);
        const Words4 b = *reinterpret_cast<const Words4 *>(static_cast<const float *>(row) + c + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(a.w[j]);
            v[4 + j] = __uint_as_float(b.w[j]);
        }
    } else {
        const Words2 a = *reinterpret_cast<const Words2 *>(static_cast<const uint16_t *>(row) + c);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = from_bits16((a.w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, kDtype);
    }
}

// The same for those below H; 0 past H.
template <int kDtype>
__device__ __forceinline__ void load8(const void *row, int c, int H, float (&v)[8])
{
    if (c + 8 <= H) {
        load8_whole<kDtype>(row, c, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0.0f;
            if (c + j < H) {
                if constexpr (kDtype == INT4VH_ROWS_F32)
                    v[j] = static_cast<const float *>(row)[c + j];
                else
                    v[j] = from_bits16(static_cast<const uint16_t *>(row)[c + j], kDtype);
            }
        }
    }
}

__device__ __forceinline__ void load8_any(const void *row, int dtype, int c, int H, float (&v)[8])
{
    if (dtype == INT4VH_ROWS_F16)
        load8<INT4VH_ROWS_F16>(row, c, H, v);
    else if (dtype == INT4VH_ROWS_BF16)
        load8<INT4VH_ROWS_BF16>(row, c, H, v);
    else
        load8<INT4VH_ROWS_F32>(row, c, H, v);
}

// The one rounding of each value to the output's type.
__device__ __forceinline__ void store8(void *row, int dtype, int c, int H, const float (&v)[8])
{
    if (dtype == INT4VH_ROWS_F32) {
        float *p = static_cast<float *>(row) + c;
        if (c + 8 <= H) {
            Words4 a, b;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a.w[j] = __float_as_uint(v[j]);
                b.w[j] = __float_as_uint(v[4 + j]);
            }
            *reinterpret_cast<Words4 *>(p) = a;
            *reinterpret_cast<Words4 *>(p + 4) = b;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < H)
                    p[j] = v[j];
        }
        return;
    }
    uint16_t *p = static_cast<uint16_t *>(row) + c;
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        u[j] = to_bits16(v[j], dtype);
    if (c + 8 <= H) {
        Words2 a;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a.w[j] = u[2 * j] | (u[2 * j + 1] << 16);
        *reinterpret_cast<Words2 *>(p) = a;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < H)
                p[j] = (uint16_t)u[j];
    }
}

__device__ __forceinline__ void store_codes8(int8_t *p, int c, int H, const int (&q)[8])
{
    if (c + 8 <= H) {
        Pair1 a;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            a.w[j] = (q[4 * j] & 0xFF) | ((q[4 * j + 1] & 0xFF) << 8) | ((q[4 * j + 2] & 0xFF) << 16) |
                     ((uint32_t)q[4 * j + 3] << 24);
        *reinterpret_cast<Pair1 *>(p + c) = a;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < H)
                p[c + j] = (int8_t)q[j];
    }
}

// Sum and largest word over each kLanes lanes, the same in all of them.
template <int kLanes, bool kSum, bool kPeak>
__device__ __forceinline__ void reduce(float &ss, uint32_t &peak)
{
#pragma unroll
    for (int off = kLanes / 2; off >= 1; off >>= 1) {
        if (kSum)
            ss += __shfl_xor(ss, off);
        if (kPeak) {
            const uint32_t o = __shfl_xor(peak, off);
            peak = o > peak ? o : peak;
        }
    }
}

// Grid: workgroups over rows, a thread for every 8 channels.  kInt8: the 8-bit
// output; kNorm: divide by the root mean square.
template <int kDtype, bool kInt8, bool kNorm>
__global__ void __launch_bounds__(kMaxThreads) norm_rows_kernel(NormArgs a)
{
    __shared__ float s_sum[2][kMaxThreads / 64];
    __shared__ uint32_t s_peak[2][kMaxThreads / 64];
    __shared__ float s_again[kMaxThreads / 64];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, wave = tid >> 6, n_waves = nt >> 6;
    const int H = a.H;
    constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;
    const size_t out_size = a.out_dtype == INT4VH_ROWS_F32 ? 4 : 2;

    const int c = 8 * tid;                     // this thread's first channel
    float w[8], cs[8];
    if (kNorm)
        load8_any(a.weight, a.weight_dtype, c, H, w);
    if (kInt8) {
        if (a.channel) {
            load8<INT4VH_ROWS_F16>(a.channel, c, H, cs);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                cs[j] = 1.0f;
        }
    }

    // sums of squares that serve as they are
    const float low_sum = a.eps < kLowMean ? kLowMean * (float)H : 0.0f;
    const float high_sum = a.eps < 0x1p126f ? 0x1p127f : 0.0f;

    int buf = 0;
    for (unsigned m = blockIdx.x; m < (unsigned)a.M; m += gridDim.x, buf ^= 1) {
        float h[8];
        load8<kDtype>(static_cast<const char *>(a.x) + (size_t)m * a.x_stride * kSize, c, H, h);
        if (a.residual) {
            float r[8];
            load8<kDtype>(static_cast<const char *>(a.residual) + (size_t)m * a.residual_stride * kSize, c, H, r);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[j] += r[j];
            if (a.sum_out)
                store8(static_cast<char *>(a.sum_out) + (size_t)m * H * kSize, kDtype, c, H, h);
        }
        float t[8];                            // what 8 bits stand for, up to rstd
        if (kInt8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                t[j] = (kNorm ? h[j] * w[j] : h[j]) * cs[j];
        }

        // one reduction: the sum of squares, and the largest |t| as an
        // unsigned word (a NaN is above infinity, which is above every number)
        float ss = 0.0f;
        uint32_t peak = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (kNorm)
                ss = __builtin_fmaf(h[j], h[j], ss);
            if (kInt8) {
                const uint32_t u = __float_as_uint(t[j]) & 0x7FFFFFFFu;
                peak = u > peak ? u : peak;
            }
        }
        reduce<64, kNorm, kInt8>(ss, peak);
        if (n_waves > 1) {
            if (lane == 0) {
                s_sum[buf][wave] = ss;
                s_peak[buf][wave] = peak;
            }
            // the other half of the arrays is the next row's, so one barrier a row
            __syncthreads();
            const int i = lane & 15;
            ss = i < n_waves ? s_sum[buf][i] : 0.0f;
            peak = i < n_waves ? s_peak[buf][i] : 0u;
            reduce<16, kNorm, kInt8>(ss, peak);
        }
        const float pk = __uint_as_float(peak);
        const bool tiny = pk < kTinyPeak;
        if (kInt8) {
            const bool live = !tiny && peak < 0x7F800000u;
            const float inv = 127.0f / pk;
            int q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)        // |t * inv| <= 127 (1 + 2^-23): rint never leaves [-127, 127]
                q[j] = live ? (int)rintf(t[j] * inv) : 0;
            store_codes8(a.codes + (size_t)m * H, c, H, q);
        }
        // before and behind: powers of two that make up for another scale
        float eps = a.eps, before = 1.0f, behind = 1.0f;
        // The same in every thread: a scalar, for a jump out of the usual way.
        // binary16 rows stay inside by far (between 2^-48 and 2^47).
        const bool again = kNorm && kDtype != INT4VH_ROWS_F16 &&
                           __builtin_amdgcn_readfirstlane(ss < low_sum || ss > high_sum);
        if (__builtin_expect(again, false)) {
            const bool low = ss < low_sum;
            const float f = low ? kUp : kDown;
            ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = __builtin_fmaf(h[j] * f, h[j] * f, ss);
            uint32_t none = 0u;
            reduce<64, true, false>(ss, none);
            if (n_waves > 1) {
                if (lane == 0)
                    s_again[wave] = ss;        // the row before read it in front of this row's first barrier
                __syncthreads();
                ss = (lane & 15) < n_waves ? s_again[lane & 15] : 0.0f;
                reduce<16, true, false>(ss, none);
            }
            eps = eps * f * f;
            // small rows are scaled up front, large ones at the end: no
            // product in between overflows or loses bits
            before = low ? f : 1.0f;
            behind = low ? 1.0f : f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[j] *= before;
        }
        if (kInt8) {
            if (tid == 0) {
                const float rstd = kNorm ? 1.0f / sqrtf(ss / (float)H + eps) : 1.0f;
                float top = pk * rstd;
                if (__builtin_expect(again, false))    // exact in binary64, then the product's one rounding
                    top = (float)((double)pk * rstd * before * behind);
                a.row_scales[m] = tiny ? 0.0f : top / 127.0f;
            }
        } else {
            const float rstd = 1.0f / sqrtf(ss / (float)H + eps);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = h[j] * rstd * behind * w[j];
            store8(static_cast<char *>(a.out) + (size_t)m * H * out_size, a.out_dtype, c, H, y);
        }
    }
}

// Rows of more than 8192 channels in 8 bits (the inputs of wide linear layers):
// kChunks chunks of 8 channels per thread, still read once and held in
// registers.  A chunk that would pass the row's end takes the last 8 channels,
// so that all loads are alike and in flight together; what two threads hold
// both, both write, with the same value.  Measured (graph-timed): 4096 x 25600
// bfloat16 rows 77 us (4.1 TB/s), 4096 x 16384 44 us (4.6), 16 x 25600 4.9 us.
template <int kDtype, int kChunks>
__global__ void __launch_bounds__(kMaxThreads) quantize_long_kernel(NormArgs a)
{
    __shared__ uint32_t s_peak[2][kMaxThreads / 64];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, wave = tid >> 6, n_waves = nt >> 6;
    const int H = a.H;
    constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;
    int buf = 0;
    for (unsigned m = blockIdx.x; m < (unsigned)a.M; m += gridDim.x, buf ^= 1) {
        const char *row = static_cast<const char *>(a.x) + (size_t)m * a.x_stride * kSize;
        float t[kChunks][8];
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            load8_whole<kDtype>(row, min(8 * (tid + i * nt), H - 8), t[i]);
        if (a.channel) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                float cs[8];
                load8_whole<INT4VH_ROWS_F16>(a.channel, min(8 * (tid + i * nt), H - 8), cs);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    t[i][j] *= cs[j];
            }
        }
        float none = 0.0f;
        uint32_t peak = 0u;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = __float_as_uint(t[i][j]) & 0x7FFFFFFFu;
                peak = u > peak ? u : peak;
            }
        reduce<64, false, true>(none, peak);
        if (lane == 0)
            s_peak[buf][wave] = peak;
        __syncthreads();                       // the other half of the array is the next row's
        peak = (lane & 15) < n_waves ? s_peak[buf][lane & 15] : 0u;
        reduce<16, false, true>(none, peak);
        const float pk = __uint_as_float(peak);
        const bool tiny = pk < kTinyPeak;
        const bool live = !tiny && peak < 0x7F800000u;
        const float inv = 127.0f / pk;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            int q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = live ? (int)rintf(t[i][j] * inv) : 0;
            store_codes8(a.codes + (size_t)m * H, min(8 * (tid + i * nt), H - 8), H, q);
        }
        if (tid == 0)
            a.row_scales[m] = tiny ? 0.0f : pk / 127.0f;
    }
}

template <int kDtype, int kChunks>
int launch_long(const NormArgs &a, hipStream_t s)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e, "hipGetDevice");
    const int nt = (a.H + 512 * kChunks - 1) / (512 * kChunks) * 64;
    const int resident = cu_count(dev) * (2048 / nt);
    const int grid = a.M < resident ? a.M : resident;
    hipLaunchKernelGGL((quantize_long_kernel<kDtype, kChunks>), dim3(grid), dim3(nt), 0, s, a);
    e = hipGetLastError();
    return e == hipSuccess ? INT4VH_OK : hip_fail(e, "row quantisation kernel launch");
}

// The fewest chunks per thread that 1024 threads can hold the row with.
template <int kDtype>
int launch_long_rows(const NormArgs &a, hipStream_t s)
{
    if (a.H <= 2 * INT4VH_MAX_H)
        return launch_long<kDtype, 2>(a, s);
    return a.H <= 4 * INT4VH_MAX_H ? launch_long<kDtype, 4>(a, s) : launch_long<kDtype, 8>(a, s);
}

template <int kDtype, bool kInt8, bool kNorm>
int launch_rows(const NormArgs &a, hipStream_t s)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e, "hipGetDevice");
    const int nt = (a.H + 511) / 512 * 64;
    const int resident = cu_count(dev) * (2048 / nt);
    const int grid = a.M < resident ? a.M : resident;
    hipLaunchKernelGGL((norm_rows_kernel<kDtype, kInt8, kNorm>), dim3(grid), dim3(nt), 0, s, a);
    e = hipGetLastError();
    return e == hipSuccess ? INT4VH_OK : hip_fail(e, "norm kernel launch");
}

template <bool kInt8, bool kNorm>
int launch(const NormArgs &a, int dtype, hipStream_t s)
{
    if (dtype == INT4VH_ROWS_F16)
        return launch_rows<INT4VH_ROWS_F16, kInt8, kNorm>(a, s);
    if (dtype == INT4VH_ROWS_BF16)
        return launch_rows<INT4VH_ROWS_BF16, kInt8, kNorm>(a, s);
    return launch_rows<INT4VH_ROWS_F32, kInt8, kNorm>(a, s);
}

// What every entry point checks of its rows.
int check_rows(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, int dtype, int M, int H,
               const void *sum_out, int max_h)
{
    if (M < 1 || H < 1 || !rows_known(dtype) || !x || (sum_out && !residual))
        return INT4VH_EINVAL;
    if (M > 1 && (x_stride < H || (residual && residual_stride < H)))
        return INT4VH_EINVAL;
    if (!rows_aligned(x, rows_size(dtype)) || !rows_aligned(residual, rows_size(dtype)) || !rows_aligned(sum_out, rows_size(dtype)))
        return INT4VH_EALIGN;
    return H > max_h ? INT4VH_EUNSUPPORTED : INT4VH_OK;
}

} // namespace

extern "C" {

int rms_norm_rows(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, int dtype,
                  const void *weight, int weight_dtype, int M, int H, float eps, void *sum_out, void *out,
                  int out_dtype, void *stream)
{
    if (!rows_known(weight_dtype) || !rows_known(out_dtype) || !weight || !out || !(eps >= 0.0f) || !std::isfinite(eps))
        return INT4VH_EINVAL;
    const int st = check_rows(x, x_stride, residual, residual_stride, dtype, M, H, sum_out, INT4VH_MAX_H);
    if (st == INT4VH_EINVAL)
        return st;
    if (!rows_aligned(weight, rows_size(weight_dtype)) || !rows_aligned(out, rows_size(out_dtype)))
        return INT4VH_EALIGN;
    if (st != INT4VH_OK)
        return st;
    const NormArgs a = {x,       residual, x_stride, residual_stride, weight, nullptr,      sum_out,
                        out,     nullptr,  nullptr,  M,               H,      weight_dtype, out_dtype,
                        eps};
    return launch<false, true>(a, dtype, static_cast<hipStream_t>(stream));
}

int rms_norm_rows_int8(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, int dtype,
                       const void *weight, int weight_dtype, const void *channel_scales, int M, int H, float eps,
                       void *sum_out, int8_t *codes, float *row_scales, void *stream)
{
    if (!rows_known(weight_dtype) || !weight || !codes || !row_scales || !(eps >= 0.0f) || !std::isfinite(eps))
        return INT4VH_EINVAL;
    const int st = check_rows(x, x_stride, residual, residual_stride, dtype, M, H, sum_out, INT4VH_MAX_H);
    if (st == INT4VH_EINVAL)
        return st;
    if (!rows_aligned(weight, rows_size(weight_dtype)) || !rows_aligned(channel_scales, 2) || !rows_aligned(row_scales, 4))
        return INT4VH_EALIGN;
    if (st != INT4VH_OK)
        return st;
    const NormArgs a = {x,       residual, x_stride,   residual_stride, weight, static_cast<const uint16_t *>(channel_scales),
                        sum_out, nullptr,  codes,      row_scales,      M,      H,
                        weight_dtype, INT4VH_ROWS_F16, eps};
    return launch<true, true>(a, dtype, static_cast<hipStream_t>(stream));
}

int quantize_rows_int8(const void *x, int64_t x_stride, int dtype, const void *channel_scales, int M, int H,
                       int8_t *codes, float *row_scales, void *stream)
{
    if (!codes || !row_scales)
        return INT4VH_EINVAL;
    const int st = check_rows(x, x_stride, nullptr, 0, dtype, M, H, nullptr, kMaxLong);
    if (st == INT4VH_EINVAL)
        return st;
    if (!rows_aligned(channel_scales, 2) || !rows_aligned(row_scales, 4))
        return INT4VH_EALIGN;
    if (st != INT4VH_OK)
        return st;
    const NormArgs a = {x,       nullptr, x_stride, 0, nullptr, static_cast<const uint16_t *>(channel_scales),
                        nullptr, nullptr, codes,    row_scales, M, H,
                        INT4VH_ROWS_F16, INT4VH_ROWS_F16, 0.0f};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (H <= INT4VH_MAX_H)
        return launch<true, false>(a, dtype, s);
    if (dtype == INT4VH_ROWS_F16)
        return launch_long_rows<INT4VH_ROWS_F16>(a, s);
    return dtype == INT4VH_ROWS_BF16 ? launch_long_rows<INT4VH_ROWS_BF16>(a, s) : launch_long_rows<INT4VH_ROWS_F32>(a, s);
}

} // extern "C"
