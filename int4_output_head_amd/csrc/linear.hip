// linear.hip -- 8-bit activations times packed int4 weights with a fused
// epilogue, for MI355X (gfx950): the linear layers whose weights have the
// output head's format (formulas and order of rounding in int4vh_linear.h).
//
// Nibbles become int8 operands of v_mfma_i32_16x16x64_i8 without a table: a
// nibble moved to the high half of its byte is 16*q, so a packed word gives
// the even channels by (w << 4) & 0xF0F0F0F0 and the odd ones by
// w & 0xF0F0F0F0; the factor 16 leaves exactly with the row's scale.  The
// activations' bytes are put into the same order (even channels, then odd
// ones, within every 8).  All sums are exact in int32: |16 * acc| <=
// 128 * 128 * K <= 2^30 for K <= 65536.
//
// Two kernels.  Up to 32 rows the call is the weights' stream (N * K / 2
// bytes): linear_stream_kernel gives each wave a slice of K whose activations
// stay in its registers, loads a tile of 16 weight rows per workgroup
// straight into registers with every load in flight, and adds the waves'
// exact sums through LDS.  Beyond, linear_tile_kernel is a tiled product,
// bound by the int8 matrix cores: weights stay packed until the wave that
// multiplies them has them in registers, so LDS moves half the bytes of an
// int8 tile.  Where a product has too few tiles to fill the card, its sum over
// K is split and the int32 parts are added by linear_join_kernel.
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>

#include "int4vh.h"
#include "int4vh_internal.h"
#include "int4vh_linear.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace {

using namespace int4vh_detail;

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaitLgkm0 = 0xF | (0x3 << 14) | (0x7 << 4);
constexpr uint32_t kHigh = 0xF0F0F0F0u;

struct LinArgs {
    const int8_t *codes;       // [M, K], rows codes_stride apart
    long long codes_stride;
    const float *row_scales;   // [M]
    const uint8_t *w;          // [N, K/2]
    const float *out_scales;   // [N] or null
    const void *bias;          // [N] of dtype, or null
    const void *residual;      // rows residual_stride apart, or null
    long long residual_stride;
    void *out;                 // rows out_stride apart
    long long out_stride;
    int32_t *parts;            // [splits, M, n_pad] partial sums, or null
    int M, N, K;
    int n_pad;                 // N rounded up to 4
    int activation, dtype;
    int splits, split_units;   // parts of K, and units of 128 channels in each
    int tiles_m, tiles_n;
};

__device__ __forceinline__ void barrier_no_fence()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 32 consecutive activation bytes -> the two operands (channels 0-15 and
// 16-31), even channels before odd ones within every 8
__device__ __forceinline__ void order_codes(const u32x4 &lo, const u32x4 &hi, i32x4 &a0, i32x4 &a1)
{
    const uint32_t ev = 0x06040200u, od = 0x07050301u;
    a0 = i32x4{(int32_t)__builtin_amdgcn_perm(lo[1], lo[0], ev), (int32_t)__builtin_amdgcn_perm(lo[1], lo[0], od),
               (int32_t)__builtin_amdgcn_perm(lo[3], lo[2], ev), (int32_t)__builtin_amdgcn_perm(lo[3], lo[2], od)};
    a1 = i32x4{(int32_t)__builtin_amdgcn_perm(hi[1], hi[0], ev), (int32_t)__builtin_amdgcn_perm(hi[1], hi[0], od),
               (int32_t)__builtin_amdgcn_perm(hi[3], hi[2], ev), (int32_t)__builtin_amdgcn_perm(hi[3], hi[2], od)};
}

// half h (16 of 32 channels) of a packed 16-byte chunk as an operand
__device__ __forceinline__ i32x4 weight_half(const u32x4 &q, int h)
{
    return i32x4{(int32_t)((q[2 * h] << 4) & kHigh), (int32_t)(q[2 * h] & kHigh),
                 (int32_t)((q[2 * h + 1] << 4) & kHigh), (int32_t)(q[2 * h + 1] & kHigh)};
}

__device__ __forceinline__ float load_one(const void *p, size_t i, int dtype)
{
    return dtype == INT4VH_ROWS_F32 ? static_cast<const float *>(p)[i]
                                    : from_bits16(static_cast<const uint16_t *>(p)[i], dtype);
}

__device__ __forceinline__ float activate(float y, int activation)
{
    if (activation == INT4VH_ACT_RELU)
        return y < 0.0f ? 0.0f : y;      // a NaN stays one
    if (activation == INT4VH_ACT_GELU)
        return (0.5f * y) * (1.0f + erff(y * 0.70710678118654752f));
    if (activation == INT4VH_ACT_SILU)
        return y / (1.0f + expf(-y));
    return y;
}

// acc holds 16 times the exact sum; row_scale / 16 is exact, and so is the
// conversion for |acc| < 2^28 (its low four bits are zero).  Without fused
// multiply-adds, in the order of int4vh_linear.h.
__device__ __forceinline__ float scale_bias(int32_t acc, float row_scale, float out_scale, float bias, bool scaled,
                                            bool biased)
{
    float y = ((float)acc * 0.0625f) * row_scale;
    if (scaled)
        y = y * out_scale;
    if (biased)
        y = y + bias;
    return y;
}

// One output element.
__device__ __forceinline__ void finish_one(const LinArgs &a, int m, int n, int32_t acc, float row_scale,
                                           float out_scale, float bias)
{
    float y = activate(scale_bias(acc, row_scale, out_scale, bias, a.out_scales != nullptr, a.bias != nullptr),
                       a.activation);
    if (a.residual)
        y = y + load_one(a.residual, (size_t)m * a.residual_stride + n, a.dtype);
    const size_t o = (size_t)m * a.out_stride + n;
    if (a.dtype == INT4VH_ROWS_F32)
        static_cast<float *>(a.out)[o] = y;
    else
        static_cast<uint16_t *>(a.out)[o] = (uint16_t)to_bits16(y, a.dtype);
}

// Four consecutive output elements n .. n+3 of row m (n % 4 == 0).
__device__ __forceinline__ void finish_four(const LinArgs &a, int m, int n, const i32x4 &acc, float row_scale,
                                            const float (&out_scale)[4], const float (&bias)[4])
{
    if (n + 4 > a.N) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N)
                finish_one(a, m, n + r, acc[r], row_scale, out_scale[r], bias[r]);
        return;
    }
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        y[r] = activate(
            scale_bias(acc[r], row_scale, out_scale[r], bias[r], a.out_scales != nullptr, a.bias != nullptr),
            a.activation);
    const size_t o = (size_t)m * a.out_stride + n;
    if (a.residual) {
        const size_t i = (size_t)m * a.residual_stride + n;
        if (a.dtype == INT4VH_ROWS_F32) {
            const Words4 v = *reinterpret_cast<const Words4 *>(static_cast<const float *>(a.residual) + i);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y[r] += __uint_as_float(v.w[r]);
        } else {
            const Pair2 v = *reinterpret_cast<const Pair2 *>(static_cast<const uint16_t *>(a.residual) + i);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y[r] += from_bits16((v.w[r >> 1] >> (16 * (r & 1))) & 0xFFFFu, a.dtype);
        }
    }
    if (a.dtype == INT4VH_ROWS_F32) {
        Words4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v.w[r] = __float_as_uint(y[r]);
        *reinterpret_cast<Words4 *>(static_cast<float *>(a.out) + o) = v;
    } else {
        Pair2 v;
        v.w[0] = to_bits16(y[0], a.dtype) | (to_bits16(y[1], a.dtype) << 16);
        v.w[1] = to_bits16(y[2], a.dtype) | (to_bits16(y[3], a.dtype) << 16);
        *reinterpret_cast<Pair2 *>(static_cast<uint16_t *>(a.out) + o) = v;
    }
}

// out_scales and bias of columns n .. n+3 (neutral past N or where absent)
__device__ __forceinline__ void load_columns(const LinArgs &a, int n, float (&os)[4], float (&bs)[4])
{
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const bool in = n + r < a.N;
        os[r] = in && a.out_scales ? a.out_scales[n + r] : 1.0f;
        bs[r] = in && a.bias ? load_one(a.bias, n + r, a.dtype) : 0.0f;
    }
}

// ---------------------------------------------------------------- up to 32 rows
constexpr int kSWaves = 8;
constexpr int kSThreads = 64 * kSWaves;
constexpr int kSMaxUnits = 8;                         // units of 128 channels per wave
constexpr int kSMaxK = kSWaves * kSMaxUnits * 128;    // 8192 channels per workgroup

// Grid (workgroups over tiles of 16 weight rows, parts of K).  kMB: blocks of
// 16 activation rows; kUnits: units per wave.
template <int kMB, int kUnits>
__global__ void __launch_bounds__(kSThreads) linear_stream_kernel(LinArgs a)
{
    __shared__ __attribute__((aligned(16))) int32_t s_part[2][kSWaves][kMB][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n16 = lane & 15, grp = lane >> 4;
    const int k_begin = (int)blockIdx.y * a.split_units * 128;
    const int k_end = min(a.K, k_begin + a.split_units * 128);
    const int n_tiles = a.tiles_n;
    const int ch0 = k_begin + wave * (kUnits * 128) + 32 * grp;   // this lane's channels in its wave's unit 0

    const size_t row_bytes = (size_t)(a.K / 2);
    auto load_w = [&](int tile, u32x4 (&q)[kUnits]) {
        const int n = min(tile * 16 + n16, a.N - 1);
        const uint8_t *row = a.w + (size_t)n * row_bytes;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            // past the end: any valid chunk, it meets zero codes
            const int c = min(ch0 + 128 * u, a.K - 32);
            q[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row + c / 2));
        }
    };

    u32x4 q[kUnits];
    int tile = blockIdx.x;
    load_w(tile, q);

    i32x4 A[kMB][kUnits][2];
#pragma unroll
    for (int mb = 0; mb < kMB; ++mb) {
        const int m = mb * 16 + n16;
        const int8_t *row = a.codes + (size_t)min(m, a.M - 1) * a.codes_stride;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = ch0 + 128 * u;
            u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
            if (m < a.M && c < k_end) {
                lo = *reinterpret_cast<const u32x4 *>(row + c);
                hi = *reinterpret_cast<const u32x4 *>(row + c + 16);
            }
            order_codes(lo, hi, A[mb][u][0], A[mb][u][1]);
        }
    }

    for (int buf = 0; tile < n_tiles; buf ^= 1) {
        const int next = tile + gridDim.x;
        i32x4 acc[kMB];
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb)
            acc[mb] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const i32x4 w0 = weight_half(q[u], 0), w1 = weight_half(q[u], 1);
#pragma unroll
            for (int mb = 0; mb < kMB; ++mb) {
                acc[mb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, A[mb][u][0], acc[mb], 0, 0, 0);
                acc[mb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, A[mb][u][1], acc[mb], 0, 0, 0);
            }
        }
        if (next < n_tiles)
            load_w(next, q);
        // D: column = activation row lane & 15, rows = weight rows 4 * grp + r
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb)
            *reinterpret_cast<i32x4 *>(&s_part[buf][wave][mb][lane * 4]) = acc[mb];
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        barrier_no_fence();                 // the other buffer is the next tile's
        for (int o = tid; o < kMB * 256; o += kSThreads) {
            const int mb = o >> 8, m = mb * 16 + ((o >> 4) & 15), nn = o & 15;
            const int n = tile * 16 + nn;
            if (m < a.M && n < a.N) {
                const int at = ((nn >> 2) * 16 + (m & 15)) * 4 + (nn & 3);
                int32_t sum = 0;
#pragma unroll
                for (int w = 0; w < kSWaves; ++w)
                    sum += s_part[buf][w][mb][at];
                if (a.parts)
                    a.parts[((size_t)blockIdx.y * a.M + m) * a.n_pad + n] = sum;
                else
                    finish_one(a, m, n, sum, a.row_scales[m], a.out_scales ? a.out_scales[n] : 1.0f,
                               a.bias ? load_one(a.bias, n, a.dtype) : 0.0f);
            }
        }
        tile = next;
    }
}

// ---------------------------------------------------------------- tiles
// A workgroup computes kWM*kMB*16 activation rows x kWN*kNB*16 weight rows
// with kWM x kWN waves.  Per K step of 128 channels each thread brings
// 32-byte pieces of activations and 16-byte pieces of packed weights through
// registers into LDS, in fragment order (every LDS access is 1 KB contiguous
// per wave, no bank conflicts), one step ahead; two LDS buffers, one barrier a
// step.
template <int kWM, int kWN, int kMB, int kNB>
__global__ void __launch_bounds__(64 * kWM *kWN) linear_tile_kernel(LinArgs a)
{
    constexpr int kThreads = 64 * kWM * kWN;
    constexpr int kBM = kWM * kMB, kBN = kWN * kNB;           // blocks of 16
    constexpr int kAPer = kBM * 64 / kThreads, kWPer = kBN * 64 / kThreads;
    static_assert(kAPer * kThreads == kBM * 64 && kWPer * kThreads == kBN * 64, "whole pieces per thread");
    struct Lds {
        u32x4 act[kBM][2][64];
        u32x4 w[kBN][64];
    };
    __shared__ Lds lds[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n16 = lane & 15, grp = lane >> 4;
    const int wm = wave % kWM, wn = wave / kWM;

    // Workgroups are dispatched to the 8 XCDs round-robin: renumber them so
    // that each XCD takes neighbouring tiles and shares operands in its L2.
    const int total = a.tiles_m * a.tiles_n * a.splits;
    const int xcd = (int)blockIdx.x % 8, at = (int)blockIdx.x / 8, each = total / 8, more = total % 8;
    const int id = xcd * each + min(xcd, more) + at;
    const int part = id / (a.tiles_m * a.tiles_n);
    const int t = id % (a.tiles_m * a.tiles_n);
    constexpr int kGroup = 8;                                  // tiles of M that share a column of weights
    const int first = t / (kGroup * a.tiles_n) * kGroup, rows = min(kGroup, a.tiles_m - first);
    const int in = t % (kGroup * a.tiles_n);
    const int m0 = (first + in % rows) * kBM * 16, n0 = (in / rows) * kBN * 16;
    const int s0 = part * a.split_units, s1 = min(s0 + a.split_units, (a.K + 127) / 128);

    const int8_t *arow[kAPer];
    const uint8_t *wrow[kWPer];
#pragma unroll
    for (int j = 0; j < kAPer; ++j) {
        const int m = m0 + ((tid + j * kThreads) >> 6) * 16 + n16;
        arow[j] = a.codes + (size_t)min(m, a.M - 1) * a.codes_stride;
    }
#pragma unroll
    for (int j = 0; j < kWPer; ++j) {
        const int n = n0 + ((tid + j * kThreads) >> 6) * 16 + n16;
        wrow[j] = a.w + (size_t)min(n, a.N - 1) * (size_t)(a.K / 2);
    }
    u32x4 ra[kAPer][2], rw[kWPer];
    auto load = [&](int s) {
        const int c = s * 128 + 32 * grp;
        const int cc = min(c, a.K - 32);
#pragma unroll
        for (int j = 0; j < kAPer; ++j) {
            const u32x4 *p = reinterpret_cast<const u32x4 *>(arow[j] + cc);
            ra[j][0] = p[0];
            ra[j][1] = p[1];
        }
#pragma unroll
        for (int j = 0; j < kWPer; ++j)
            rw[j] = *reinterpret_cast<const u32x4 *>(wrow[j] + cc / 2);
    };
    auto store = [&](int s, Lds &l) {
        const bool live = s * 128 + 32 * grp < a.K;            // channels past K: zero codes
#pragma unroll
        for (int j = 0; j < kAPer; ++j) {
            i32x4 x0, x1;
            order_codes(ra[j][0], ra[j][1], x0, x1);
            const int b = (tid + j * kThreads) >> 6;
            l.act[b][0][lane] = __builtin_bit_cast(u32x4, live ? x0 : i32x4{0, 0, 0, 0});
            l.act[b][1][lane] = __builtin_bit_cast(u32x4, live ? x1 : i32x4{0, 0, 0, 0});
        }
#pragma unroll
        for (int j = 0; j < kWPer; ++j)
            l.w[(tid + j * kThreads) >> 6][lane] = rw[j];
    };

    i32x4 acc[kMB][kNB];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};

    load(s0);
    store(s0, lds[0]);
    for (int s = s0; s < s1; ++s) {
        const Lds &l = lds[(s - s0) & 1];
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        barrier_no_fence();
        const int sn = min(s + 1, s1 - 1);                     // the last step loads itself again, unused
        load(sn);
        u32x4 q[kNB];
#pragma unroll
        for (int j = 0; j < kNB; ++j)
            q[j] = l.w[wn * kNB + j][lane];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 x[kMB];
#pragma unroll
            for (int i = 0; i < kMB; ++i)
                x[i] = __builtin_bit_cast(i32x4, l.act[wm * kMB + i][h][lane]);
#pragma unroll
            for (int j = 0; j < kNB; ++j) {
                const i32x4 w = weight_half(q[j], h);
#pragma unroll
                for (int i = 0; i < kMB; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x[i], acc[i][j], 0, 0, 0);
            }
        }
        if (s + 1 < s1)
            store(s + 1, lds[(s + 1 - s0) & 1]);
    }

    // D: column = activation row lane & 15, rows = weight rows 4 * grp + r
    if (a.parts) {
#pragma unroll
        for (int i = 0; i < kMB; ++i) {
            const int m = m0 + (wm * kMB + i) * 16 + n16;
#pragma unroll
            for (int j = 0; j < kNB; ++j) {
                const int n = n0 + (wn * kNB + j) * 16 + 4 * grp;
                if (m < a.M && n < a.n_pad)
                    *reinterpret_cast<i32x4 *>(&a.parts[((size_t)part * a.M + m) * a.n_pad + n]) = acc[i][j];
            }
        }
        return;
    }
    float rs[kMB];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
        rs[i] = a.row_scales[min(m0 + (wm * kMB + i) * 16 + n16, a.M - 1)];
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
        const int n = n0 + (wn * kNB + j) * 16 + 4 * grp;
        float os[4], bs[4];
        load_columns(a, n, os, bs);
#pragma unroll
        for (int i = 0; i < kMB; ++i) {
            const int m = m0 + (wm * kMB + i) * 16 + n16;
            if (m < a.M && n < a.N)
                finish_four(a, m, n, acc[i][j], rs[i], os, bs);
        }
    }
}

// The parts' sums and the epilogue: one thread per four columns.
__global__ void __launch_bounds__(256) linear_join_kernel(LinArgs a)
{
    const int per_row = a.n_pad / 4;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)a.M * per_row)
        return;
    const int m = (int)(i / per_row), n = (int)(i % per_row) * 4;
    i32x4 sum = {0, 0, 0, 0};
    for (int p = 0; p < a.splits; ++p)
        sum += *reinterpret_cast<const i32x4 *>(&a.parts[((size_t)p * a.M + m) * a.n_pad + n]);
    float os[4], bs[4];
    load_columns(a, n, os, bs);
    finish_four(a, m, n, sum, a.row_scales[m], os, bs);
}

// ---------------------------------------------------------------- host side

// How a call of these sizes runs.
struct Plan {
    int kind;                  // 0: stream, 1: tiles of 256 x 256, 2: 128 x 128, 3: 64 x 128
    int splits, split_units;
    int tiles_m, tiles_n;
};

Plan plan_for(int M, int N, int K, int cus)
{
    Plan p;
    const int units = (K + 127) / 128;
    if (M <= 32) {
        p.kind = 0;
        p.tiles_m = 1;
        p.tiles_n = (N + 15) / 16;
        p.splits = (K + kSMaxK - 1) / kSMaxK;
    } else {
        const int bm[4] = {0, 256, 128, 64}, bn[4] = {0, 256, 128, 128};
        p.kind = 3;
        if (M > 64)
            p.kind = (long long)((M + 255) / 256) * ((N + 255) / 256) >= cus ? 1 : 2;
        p.tiles_m = (M + bm[p.kind] - 1) / bm[p.kind];
        p.tiles_n = (N + bn[p.kind] - 1) / bn[p.kind];
        const long long tiles = (long long)p.tiles_m * p.tiles_n;
        p.splits = 1;
        // at least 4 steps of 128 channels in a part
        while (p.splits * 2 * tiles <= 2 * cus && units / (p.splits * 2) >= 4)
            p.splits *= 2;
    }
    p.split_units = (units + p.splits - 1) / p.splits;
    p.splits = (units + p.split_units - 1) / p.split_units;
    return p;
}

size_t parts_bytes(const Plan &p, int M, int N)
{
    if (p.splits < 2)
        return 0;
    const size_t b = (size_t)p.splits * M * ((N + 3) / 4 * 4) * 4;
    return (b + 255) / 256 * 256;
}

// Compute units of the current device; without one, those of an MI355X, so
// that sizes are checked alike (a launch reports the missing device).
int current_cus()
{
    int dev = 0;
    return cu_count(hipGetDevice(&dev) == hipSuccess ? dev : -1);
}

bool sizes_ok(int M, int N, int K)
{
    return M >= 1 && N >= 1 && K >= 32 && K % 32 == 0;
}

bool sizes_supported(int M, int N, int K)
{
    return K <= 65536 && N <= (1 << 24) && M <= (1 << 20) && (long long)M * N < (1ll << 40);
}

template <int kMB>
void launch_stream(const LinArgs &a, dim3 grid, hipStream_t s)
{
    const int per_wave = (a.split_units + kSWaves - 1) / kSWaves;
    const dim3 block(kSThreads);
    if (per_wave <= 1)
        hipLaunchKernelGGL((linear_stream_kernel<kMB, 1>), grid, block, 0, s, a);
    else if (per_wave <= 2)
        hipLaunchKernelGGL((linear_stream_kernel<kMB, 2>), grid, block, 0, s, a);
    else if (per_wave <= 3)
        hipLaunchKernelGGL((linear_stream_kernel<kMB, 3>), grid, block, 0, s, a);
    else if (per_wave <= 5)
        hipLaunchKernelGGL((linear_stream_kernel<kMB, 5>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((linear_stream_kernel<kMB, 8>), grid, block, 0, s, a);
}

} // namespace

extern "C" {

size_t linear_int4_rows_workspace_bytes(int M, int N, int K)
{
    if (!sizes_ok(M, N, K) || !sizes_supported(M, N, K))
        return 0;
    return parts_bytes(plan_for(M, N, K, current_cus()), M, N);
}

int linear_int4_rows(const int8_t *codes, int64_t codes_stride, const float *row_scales, const uint8_t *packed_w,
                     const float *out_scales, const void *bias, int activation, const void *residual,
                     int64_t residual_stride, int M, int N, int K, void *out, int64_t out_stride, int dtype,
                     void *workspace, size_t workspace_bytes, void *stream)
{
    if (!sizes_ok(M, N, K) || !codes || !row_scales || !packed_w || !out || !rows_known(dtype) ||
        activation < INT4VH_ACT_NONE || activation > INT4VH_ACT_SILU)
        return INT4VH_EINVAL;
    if (M > 1 && (codes_stride < K || out_stride < N || (residual && residual_stride < N)))
        return INT4VH_EINVAL;
    const size_t el = rows_size(dtype);
    if (!rows_aligned(codes, 16) || (M > 1 && codes_stride % 16) || !rows_aligned(packed_w, 16) ||
        !rows_aligned(row_scales, 4) || !rows_aligned(out_scales, 4) || !rows_aligned(bias, el) ||
        !rows_aligned(residual, el) || !rows_aligned(out, el))
        return INT4VH_EALIGN;
    if (!sizes_supported(M, N, K))
        return INT4VH_EUNSUPPORTED;
    const int cus = current_cus();
    const Plan p = plan_for(M, N, K, cus);
    const size_t need = parts_bytes(p, M, N);
    if (need) {
        if (!workspace)
            return INT4VH_EINVAL;
        if (!rows_aligned(workspace, 256))
            return INT4VH_EALIGN;
        if (workspace_bytes < need)
            return INT4VH_EWORKSPACE;
    }
    LinArgs a;
    a.codes = codes;
    a.codes_stride = codes_stride;
    a.row_scales = row_scales;
    a.w = packed_w;
    a.out_scales = out_scales;
    a.bias = bias;
    a.residual = residual;
    a.residual_stride = residual_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.parts = need ? static_cast<int32_t *>(workspace) : nullptr;
    a.M = M;
    a.N = N;
    a.K = K;
    a.n_pad = (N + 3) / 4 * 4;
    a.activation = activation;
    a.dtype = dtype;
    a.splits = p.splits;
    a.split_units = p.split_units;
    a.tiles_m = p.tiles_m;
    a.tiles_n = p.tiles_n;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 tiles((unsigned)((long long)p.tiles_m * p.tiles_n * p.splits));
    if (p.kind == 0) {
        const dim3 grid(p.tiles_n < 2 * cus ? p.tiles_n : 2 * cus, p.splits);
        if (M <= 16)
            launch_stream<1>(a, grid, s);
        else
            launch_stream<2>(a, grid, s);
    } else if (p.kind == 1) {
        hipLaunchKernelGGL((linear_tile_kernel<4, 2, 4, 8>), tiles, dim3(512), 0, s, a);
    } else if (p.kind == 2) {
        hipLaunchKernelGGL((linear_tile_kernel<2, 2, 4, 4>), tiles, dim3(256), 0, s, a);
    } else {
        hipLaunchKernelGGL((linear_tile_kernel<1, 4, 4, 2>), tiles, dim3(256), 0, s, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return hip_fail(e, "linear kernel launch");
    if (need) {
        const long long n4 = (long long)M * (a.n_pad / 4);
        hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s, a);
        e = hipGetLastError();
        if (e != hipSuccess)
            return hip_fail(e, "linear join kernel launch");
    }
    return INT4VH_OK;
}

} // extern "C"
