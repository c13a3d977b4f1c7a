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
// Two kernels.  Up to 16 rows the call is the weights' stream (N * K / 2
// bytes): linear_stream_kernel gives each wave a slice of K whose activations
// stay in its registers, loads a tile of 16 weight rows per workgroup straight
// into registers with every load in flight, and adds the waves' exact sums
// through LDS.  Beyond, linear_tile_kernel is a tiled product, bound by the
// matrix cores and the vector instructions: weights stay packed until the wave
// that multiplies them has them in registers, so LDS moves half the bytes of an
// int8 tile.  Where a product has too few tiles to fill the card, its sum over
// K is split and the int32 parts are added by linear_join_kernel.
//
// Measured (graph-timed, operands from HBM): 4096 x 5120 x 8192 in 190 us, 1.8
// POP/s, where a library int8 product of 8192^3 reaches 2.1 on this card
// (counters: matrix cores busy 48 % of the cycles, vector instructions 48 %, LDS
// 39 %, of its cycles 1.4 % bank conflicts); 256 x 18992 x 5120 in 50 us (34, 38
// and 41 %: 596 tiles on 256 compute units; 39 us where the operands stay in the
// last-level cache); 16 x 5120 x 5120 in 9.4 us.
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

// LDS written and read by one wave alone: its accesses execute in order, so
// only the compiler has to be held back.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// 16 consecutive activation bytes as an operand: even channels before odd ones
// within every 8
__device__ __forceinline__ i32x4 order_codes(const u32x4 &c)
{
    const uint32_t ev = 0x06040200u, od = 0x07050301u;
    return i32x4{(int32_t)__builtin_amdgcn_perm(c[1], c[0], ev), (int32_t)__builtin_amdgcn_perm(c[1], c[0], od),
                 (int32_t)__builtin_amdgcn_perm(c[3], c[2], ev), (int32_t)__builtin_amdgcn_perm(c[3], c[2], od)};
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

// acc holds 16 times the exact sum; row_scale / 16 is exact, and so is the
// conversion for |acc| < 2^28 (its low four bits are zero).  Without fused
// multiply-adds, in the order of int4vh_linear.h; an absent out_scale is 1 and
// an absent bias 0, which change no value.
__device__ __forceinline__ float scale_bias(int32_t acc, float row_scale, float out_scale, float bias)
{
    return ((float)acc * 0.0625f) * row_scale * out_scale + bias;
}

__device__ __forceinline__ float column_scale(const LinArgs &a, int n)
{
    return a.out_scales ? a.out_scales[n] : 1.0f;
}
__device__ __forceinline__ float column_bias(const LinArgs &a, int n)
{
    return a.bias ? load_one(a.bias, n, a.dtype) : 0.0f;
}

// One output element.
__device__ __forceinline__ void finish_one(const LinArgs &a, int m, int n, int32_t acc, float row_scale,
                                           float out_scale, float bias)
{
    float y[1] = {scale_bias(acc, row_scale, out_scale, bias)};
    activate(y, a.activation);
    if (a.residual)
        y[0] += load_one(a.residual, (size_t)m * a.residual_stride + n, a.dtype);
    const size_t o = (size_t)m * a.out_stride + n;
    if (a.dtype == INT4VH_ROWS_F32)
        static_cast<float *>(a.out)[o] = y[0];
    else
        static_cast<uint16_t *>(a.out)[o] = (uint16_t)to_bits16(y[0], a.dtype);
}

// Four consecutive output elements n .. n+3 <= N-1 of row m; res: the
// residual's 16-bit words where `with` is set.
__device__ __forceinline__ void finish_four(const LinArgs &a, int m, int n, const i32x4 &acc, float row_scale,
                                            const float (&out_scale)[4], const float (&bias)[4], bool with,
                                            uint2 res)
{
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        y[r] = scale_bias(acc[r], row_scale, out_scale[r], bias[r]);
    activate(y, a.activation);
    if (with) {
        y[0] += from_bits16(res.x & 0xFFFFu, a.dtype);
        y[1] += from_bits16(res.x >> 16, a.dtype);
        y[2] += from_bits16(res.y & 0xFFFFu, a.dtype);
        y[3] += from_bits16(res.y >> 16, a.dtype);
    }
    const size_t o = (size_t)m * a.out_stride + n;
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

// out_scales and bias of columns n .. n+3 (neutral where absent; past N the
// last column's, unused).  Every load is in flight before one is waited for.
__device__ __forceinline__ void load_columns(const LinArgs &a, int n, float (&os)[4], float (&bs)[4])
{
    int c[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        c[r] = min(n + r, a.N - 1);
        os[r] = 1.0f;
        bs[r] = 0.0f;
    }
    if (a.out_scales)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            os[r] = a.out_scales[c[r]];
    if (a.bias) {
        if (a.dtype == INT4VH_ROWS_F32) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                bs[r] = static_cast<const float *>(a.bias)[c[r]];
        } else {
            uint32_t u[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                u[r] = static_cast<const uint16_t *>(a.bias)[c[r]];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                bs[r] = from_bits16(u[r], a.dtype);
        }
    }
}

// ---------------------------------------------------------------- up to 16 rows
constexpr int kSRows = 16;
constexpr int kSWaves = 8;
constexpr int kSThreads = 64 * kSWaves;
constexpr int kSMaxUnits = 8;                         // units of 128 channels per wave
constexpr int kSMaxK = kSWaves * kSMaxUnits * 128;    // 8192 channels per workgroup

// Grid (workgroups over tiles of 16 weight rows, parts of K); kUnits: units per
// wave.  Loads go along the rows (4 lanes a unit's 64 bytes of weights, 8 lanes
// its 128 activation bytes: the cache looks up a line per row, not per lane)
// and turn into fragments, whose lanes go along the column, in LDS of the
// wave's own, without a barrier.  Slots are exchanged by chunk, against bank
// conflicts.
template <int kUnits>
__global__ void __launch_bounds__(kSThreads, kUnits > 5 ? 2 : 4) linear_stream_kernel(LinArgs a)
{
    constexpr int kTurn = kUnits > 2 ? kUnits : 2;    // KB per wave: its weights, or one unit of activations
    __shared__ u32x4 s_turn[kSWaves][kTurn][64];
    __shared__ __attribute__((aligned(16))) int32_t s_part[2][kSWaves][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n16 = lane & 15, grp = lane >> 4;
    const int k_begin = (int)blockIdx.y * a.split_units * 128;
    const int k_end = min(a.K, k_begin + a.split_units * 128);
    const int n_tiles = a.tiles_n;
    const int ch0 = k_begin + wave * (kUnits * 128);  // this wave's first channel
    u32x4 *turn = &s_turn[wave][0][0];

    const int wr = lane >> 2, wc = lane & 3;          // row and chunk of this lane's weight loads
    const int wslot = wc * 16 + (wr ^ (2 * wc)), wread = grp * 16 + (n16 ^ (2 * grp));
    const size_t row_bytes = (size_t)(a.K / 2);
    auto load_w = [&](int tile, u32x4 (&q)[kUnits]) {
        const uint8_t *row = a.w + (size_t)min(tile * 16 + wr, a.N - 1) * row_bytes;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            // past the end: any valid chunk, it meets zero codes
            const int c = min(ch0 + 128 * u + 32 * wc, a.K - 32);
            q[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row + c / 2));
        }
    };
    u32x4 q[kUnits];
    int tile = blockIdx.x;
    load_w(tile, q);
    // the output element of this thread in every tile (the first 4 waves at
    // most), its scales and bias asked for ahead of the sums
    const int m = tid >> 4, nn = tid & 15;
    const float row_scale = a.row_scales[min(m, a.M - 1)];

    i32x4 A[kUnits][2];
    {
        const int ac = lane & 7, ar = lane >> 3;      // chunk, and row within 8, of the activation loads
        constexpr int kFly = kUnits < 4 ? kUnits : 4; // units whose loads are in flight together
#pragma unroll
        for (int u0 = 0; u0 < kUnits; u0 += kFly) {
            u32x4 raw[kFly][2];
#pragma unroll
            for (int v = 0; v < kFly; ++v)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 8 * i + ar, c = ch0 + 128 * (u0 + v) + 16 * ac;
                    raw[v][i] = u32x4{0, 0, 0, 0};
                    if (u0 + v < kUnits && r < a.M && c < k_end)
                        raw[v][i] = *reinterpret_cast<const u32x4 *>(a.codes + (size_t)r * a.codes_stride + c);
                }
#pragma unroll
            for (int v = 0; v < kFly && u0 + v < kUnits; ++v) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    turn[(ac & 1) * 64 + (ac >> 1) * 16 + ((8 * i + ar) ^ ac)] =
                        __builtin_bit_cast(u32x4, order_codes(raw[v][i]));
                wave_fence();
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    A[u0 + v][h] = __builtin_bit_cast(i32x4, turn[h * 64 + grp * 16 + (n16 ^ (2 * grp + h))]);
                wave_fence();
            }
        }
    }

    for (int buf = 0; tile < n_tiles; buf ^= 1) {
        const int next = tile + gridDim.x, n = tile * 16 + nn;
        const float os = column_scale(a, min(n, a.N - 1)), bs = column_bias(a, min(n, a.N - 1));
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            turn[u * 64 + wslot] = q[u];
        wave_fence();
        if (next < n_tiles)
            load_w(next, q);
        i32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const u32x4 f = turn[u * 64 + wread];
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(weight_half(f, 0), A[u][0], acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(weight_half(f, 1), A[u][1], acc, 0, 0, 0);
        }
        wave_fence();
        // D: column = activation row lane & 15, rows = weight rows 4 * grp + r
        *reinterpret_cast<i32x4 *>(&s_part[buf][wave][lane * 4]) = acc;
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        barrier_no_fence();                 // the other buffer is the next tile's
        if (m < a.M && n < a.N) {
            const int at = ((nn >> 2) * 16 + m) * 4 + (nn & 3);
            int32_t sum = 0;
#pragma unroll
            for (int w = 0; w < kSWaves; ++w)
                sum += s_part[buf][w][at];
            if (a.parts)
                a.parts[((size_t)blockIdx.y * a.M + m) * a.n_pad + n] = sum;
            else
                finish_one(a, m, n, sum, row_scale, os, bs);
        }
        tile = next;
    }
}

// ---------------------------------------------------------------- tiles
// A workgroup computes kWM*kMB*16 activation rows x kWN*kNB*16 weight rows
// with kWM x kWN waves.  Per K step of 128 channels each thread brings 16-byte
// chunks of activations and packed weights through registers into LDS, one
// step ahead (two LDS buffers, one barrier a step); 8 (4) consecutive lanes
// load a row's 128 (64) bytes, since a load costs the cache a lookup per line
// and 16 lanes.  LDS holds fragments: chunk c of row r of a block of 16 rows
// lies in group c, slot r ^ x(c), which spreads both the writes (lanes along a
// row) and the reads (lanes along a column) over the banks (conflicts: 1.5 % of
// the LDS cycles of a whole call).
template <int kWM, int kWN, int kMB, int kNB, int kPerCu, int kDepth>
__global__ void __launch_bounds__(64 * kWM *kWN, kWM *kWN *kPerCu / 4) linear_tile_kernel(LinArgs a)
{
    constexpr int kThreads = 64 * kWM * kWN;
    constexpr int kBM = kWM * kMB, kBN = kWN * kNB;           // blocks of 16
    constexpr int kAPer = kBM * 128 / kThreads, kWPer = kBN * 64 / kThreads;
    static_assert(kAPer * kThreads == kBM * 128 && kWPer * kThreads == kBN * 64, "whole chunks per thread");
    struct Lds {
        u32x4 act[kBM][2][64];
        u32x4 w[kBN][64];
    };
    // the epilogue's use of LDS (per wave: 16 rows of sums and of residuals)
    constexpr int kCols = kNB * 16, kPitch = kCols + 4;        // the pitch spreads the rows over the banks
    constexpr int kRest = kCols / 2 + 2, kArea = 16 * (kPitch + kRest);
    constexpr size_t kTurn = sizeof(int32_t) * kWM * kWN * kArea;
    __shared__ __attribute__((aligned(16))) uint8_t mem[2 * sizeof(Lds) > kTurn ? 2 * sizeof(Lds) : kTurn];
    Lds *lds = reinterpret_cast<Lds *>(mem);
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

    // Rows past the end load the last one (never stored).  Addresses are a
    // uniform base, advanced by the step, and a 32-bit offset per chunk.
    const int ac = tid & 7, wc = tid & 3;                      // this thread's chunk of its rows
    const uint8_t *abase = reinterpret_cast<const uint8_t *>(a.codes) + (size_t)m0 * a.codes_stride;
    const uint8_t *wbase = a.w + (size_t)n0 * (size_t)(a.K / 2);
    uint32_t aoff[kAPer], woff[kWPer];
    int aslot[kAPer], wslot[kWPer];
#pragma unroll
    for (int j = 0; j < kAPer; ++j) {
        const int r = (tid + j * kThreads) >> 3;
        aoff[j] = (uint32_t)min(r, a.M - 1 - m0) * (uint32_t)a.codes_stride + 16u * ac;
        aslot[j] = ((r >> 4) * 2 + (ac & 1)) * 64 + (ac >> 1) * 16 + ((r & 15) ^ ac);
    }
#pragma unroll
    for (int j = 0; j < kWPer; ++j) {
        const int r = (tid + j * kThreads) >> 2;
        woff[j] = (uint32_t)min(r, a.N - 1 - n0) * (uint32_t)(a.K / 2) + 16u * wc;
        wslot[j] = (r >> 4) * 64 + wc * 16 + ((r & 15) ^ (2 * wc));
    }
    // kDepth steps are on their way in registers.  Loads past the last step
    // repeat it, and chunks past K load the row's last one, so that every step
    // issues the same loads without a branch; the codes past K are cleared on
    // their way to LDS.
    u32x4 ra[kDepth][kAPer], rw[kDepth][kWPer];
    auto load = [&](int d, int step) {
        const int s = min(step, s1 - 1);
        const uint8_t *pa = abase + (size_t)s * 128, *pw = wbase + (size_t)s * 64;
        const uint32_t backa = (uint32_t)max(0, s * 128 + 16 * ac - (a.K - 16));
        const uint32_t backw = (uint32_t)max(0, s * 64 + 16 * wc - (a.K / 2 - 16));
#pragma unroll
        for (int j = 0; j < kAPer; ++j)
            ra[d][j] = *reinterpret_cast<const u32x4 *>(pa + (aoff[j] - backa));
#pragma unroll
        for (int j = 0; j < kWPer; ++j)
            rw[d][j] = *reinterpret_cast<const u32x4 *>(pw + (woff[j] - backw));
    };
    auto store = [&](int d, int s, Lds &l) {
        if (s * 128 + 128 > a.K) {
            const bool live = s * 128 + 16 * ac < a.K;
#pragma unroll
            for (int j = 0; j < kAPer; ++j)
                ra[d][j] = live ? ra[d][j] : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < kAPer; ++j)
            (&l.act[0][0][0])[aslot[j]] = __builtin_bit_cast(u32x4, order_codes(ra[d][j]));
#pragma unroll
        for (int j = 0; j < kWPer; ++j)
            (&l.w[0][0])[wslot[j]] = rw[d][j];
    };

    i32x4 acc[kMB][kNB];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};

    const int rslot[2] = {grp * 16 + (n16 ^ (2 * grp)), grp * 16 + (n16 ^ (2 * grp + 1))};
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        load(d, s0 + d);
    store(0, s0, lds[0]);
    auto step = [&](const Lds &l) {
        u32x4 q[kNB];
#pragma unroll
        for (int j = 0; j < kNB; ++j)
            q[j] = l.w[wn * kNB + j][rslot[0]];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 x[kMB];
#pragma unroll
            for (int i = 0; i < kMB; ++i)
                x[i] = __builtin_bit_cast(i32x4, l.act[wm * kMB + i][h][rslot[h]]);
#pragma unroll
            for (int j = 0; j < kNB; ++j) {
                const i32x4 w = weight_half(q[j], h);
#pragma unroll
                for (int i = 0; i < kMB; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x[i], acc[i][j], 0, 0, 0);
            }
        }
    };
    constexpr int kTurns = kDepth % 2 ? 2 * kDepth : kDepth;   // steps after which buffers and registers repeat
    for (int s = s0; s < s1; s += kTurns) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            if (s + i >= s1)
                break;
            __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
            barrier_no_fence();
            load(i % kDepth, s + i + kDepth);
            step(lds[i & 1]);
            store((i + 1) % kDepth, s + i + 1, lds[(i + 1) & 1]);
        }
    }

    // D: column = activation row lane & 15, rows = weight rows 4 * grp + r.
    // Each wave turns its sums around in LDS, 16 activation rows at a time, so
    // that its lanes hold four columns of a row and rows are written whole.
    // The residual passes through LDS as well, loaded before anything is
    // stored: a wait for a load also waits for the stores in front of it.
    int32_t *turn = reinterpret_cast<int32_t *>(mem) + wave * kArea;
    uint32_t *rest = reinterpret_cast<uint32_t *>(turn + 16 * kPitch);
    constexpr int kLanes = kCols / 4, kStep = 64 / kLanes, kIter = 16 / kStep;   // lanes of a row; rows at a time
    const int c4 = (lane % kLanes) * 4, n = n0 + wn * kCols + c4, r0 = lane / kLanes;
    const int mw = m0 + wm * kMB * 16;
    static_assert(kMB <= 8, "two registers hold a wave's row scales");
    float os[4], bs[4], rs0 = 0.0f, rs1 = 0.0f;
    Pair2 res[kMB][kIter];
    // The usual case handles four columns at a time, with a 16-bit residual or
    // none; rows that end inside a lane's four columns, and binary32 residuals,
    // go element by element.
    const bool wide = !a.parts && a.N % 4 == 0 && (!a.residual || a.dtype != INT4VH_ROWS_F32);
    const bool early = wide && a.residual;
    if (!a.parts) {
        load_columns(a, n, os, bs);
        rs0 = a.row_scales[min(mw + lane, a.M - 1)];
        rs1 = a.row_scales[min(mw + 64 + lane, a.M - 1)];
        if (early)
#pragma unroll
            for (int i = 0; i < kMB; ++i)
#pragma unroll
                for (int k = 0; k < kIter; ++k) {
                    const int m = min(mw + i * 16 + r0 + k * kStep, a.M - 1);
                    res[i][k] = *reinterpret_cast<const Pair2 *>(static_cast<const uint16_t *>(a.residual) +
                                                                 (size_t)m * a.residual_stride + min(n, a.N - 4));
                }
    }
    // nothing below loads from memory in the usual case: a wait for a load
    // would also wait for the stores in front of it
    __builtin_amdgcn_s_waitcnt(0);
    barrier_no_fence();                                        // the last step's reads are done
#pragma unroll
    for (int i = 0; i < kMB; ++i) {
        const int mi = mw + i * 16;
#pragma unroll
        for (int j = 0; j < kNB; ++j)
            *reinterpret_cast<i32x4 *>(turn + n16 * kPitch + j * 16 + 4 * grp) = acc[i][j];
        if (early)
#pragma unroll
            for (int k = 0; k < kIter; ++k)
                *reinterpret_cast<uint2 *>(rest + (r0 + k * kStep) * kRest + c4 / 2) =
                    make_uint2(res[i][k].w[0], res[i][k].w[1]);
        wave_fence();
        const float rsi = i < 4 ? rs0 : rs1;
        if (wide) {
#pragma nounroll
            for (int r = r0; r < 16; r += kStep) {
                const i32x4 v = *reinterpret_cast<const i32x4 *>(turn + r * kPitch + c4);
                const uint2 rv = *reinterpret_cast<const uint2 *>(rest + r * kRest + c4 / 2);
                const float row_scale = __shfl(rsi, (i & 3) * 16 + r);
                if (mi + r < a.M && n < a.N)
                    finish_four(a, mi + r, n, v, row_scale, os, bs, early, rv);
            }
        } else if (a.parts) {
#pragma nounroll
            for (int r = r0; r < 16; r += kStep)
                if (mi + r < a.M && n < a.N)
                    *reinterpret_cast<i32x4 *>(&a.parts[((size_t)part * a.M + mi + r) * a.n_pad + n]) =
                        *reinterpret_cast<const i32x4 *>(turn + r * kPitch + c4);
        } else {
#pragma nounroll
            for (int e = lane; e < 16 * kCols; e += 64) {
                const int m = mi + e / kCols, c = n0 + wn * kCols + e % kCols;
                if (m < a.M && c < a.N)
                    finish_one(a, m, c, turn[e / kCols * kPitch + e % kCols], a.row_scales[m],
                               column_scale(a, c), column_bias(a, c));
            }
        }
        wave_fence();
    }
}

// The parts' sums and the epilogue: one thread per element.
__global__ void __launch_bounds__(256) linear_join_kernel(LinArgs a)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)a.M * a.N)
        return;
    const int m = (int)(i / a.N), n = (int)(i % a.N);
    int32_t sum = 0;
    for (int p = 0; p < a.splits; ++p)
        sum += a.parts[((size_t)p * a.M + m) * a.n_pad + n];
    finish_one(a, m, n, sum, a.row_scales[m], column_scale(a, n), column_bias(a, n));
}

// ---------------------------------------------------------------- host side

// How a call of these sizes runs.
enum Kind { kStream, kTile32, kTile64, kTile128 };   // tiles of 32, 64, 128 rows x 128 columns
struct Plan {
    Kind kind;
    int splits, split_units;
    int tiles_m, tiles_n;
};

long long tiles_of(int M, int N, int bm)
{
    return (long long)((M + bm - 1) / bm) * ((N + 127) / 128);
}

// Larger tiles reuse more of what they load, smaller ones fill more compute
// units.  Measured (graph-timed, us; M x N x K with tiles of 128 / 64 / 32
// rows everywhere): 4096x5120x8192 190 / 216 / 290; 4096x4096x4096 88 / 98 /
// 129; 1024x5120x5120 50 / 45 / 55; 256x18992x5120 52 / 48 / 58; 512x5120x5120
// 37 / 31 / 32; 256x5120x5120 36 / 25 / 23; 65x18992x5120 40 / 36 / 29;
// 64x5120x5120 35 / 25 / 14.  Splitting K for tiles of 32 rows, at up to two
// workgroups a compute unit, without and with: 64x5120x5120 18.3 and 14.5,
// 33x5120x5120 18.2 and 13.0, 100x300x8000 25.3 and 9.6.  16 rows in the
// stream 9.4, 17 in tiles 12.5 (5120 x 5120).
Plan plan_for(int M, int N, int K, int cus)
{
    Plan p;
    const int units = (K + 127) / 128;
    p.splits = 1;
    if (M <= kSRows) {
        p.kind = kStream;
        p.tiles_m = 1;
        p.tiles_n = (N + 15) / 16;
        p.splits = (K + kSMaxK - 1) / kSMaxK;
    } else {
        p.kind = 2 * tiles_of(M, N, 128) >= 5ll * cus  ? kTile128
                 : 4 * tiles_of(M, N, 64) >= 5ll * cus ? kTile64
                                                       : kTile32;
        const int bm = p.kind == kTile128 ? 128 : p.kind == kTile64 ? 64 : 32;
        p.tiles_m = (M + bm - 1) / bm;
        p.tiles_n = (N + 127) / 128;
        // few tiles: parts of at least 4 units, up to two workgroups a compute unit
        if (p.kind == kTile32)
            while (2 * p.splits * tiles_of(M, N, 32) <= 2ll * cus && units / (2 * p.splits) >= 4)
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

void launch_stream(const LinArgs &a, dim3 grid, hipStream_t s)
{
    const int per_wave = (a.split_units + kSWaves - 1) / kSWaves;
    const dim3 block(kSThreads);
    if (per_wave <= 1)
        hipLaunchKernelGGL(linear_stream_kernel<1>, grid, block, 0, s, a);
    else if (per_wave <= 2)
        hipLaunchKernelGGL(linear_stream_kernel<2>, grid, block, 0, s, a);
    else if (per_wave <= 3)
        hipLaunchKernelGGL(linear_stream_kernel<3>, grid, block, 0, s, a);
    else if (per_wave <= 5)
        hipLaunchKernelGGL(linear_stream_kernel<5>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(linear_stream_kernel<8>, grid, block, 0, s, a);
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
    if (!sizes_supported(M, N, K) || (M > 1 && codes_stride >= (1ll << 24)))   // a tile's chunks have 32-bit offsets
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
    if (p.kind == kStream)
        launch_stream(a, dim3(p.tiles_n < 2 * cus ? p.tiles_n : 2 * cus, p.splits), s);
    else if (p.kind == kTile32)
        hipLaunchKernelGGL((linear_tile_kernel<1, 4, 2, 2, 4, 3>), tiles, dim3(256), 0, s, a);
    else if (p.kind == kTile64)
        hipLaunchKernelGGL((linear_tile_kernel<1, 4, 4, 2, 4, 2>), tiles, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((linear_tile_kernel<2, 2, 4, 4, 2, 2>), tiles, dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return hip_fail(e, "linear kernel launch");
    if (need) {
        const long long n1 = (long long)M * N;
        hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)((n1 + 255) / 256)), dim3(256), 0, s, a);
        e = hipGetLastError();
        if (e != hipSuccess)
            return hip_fail(e, "linear join kernel launch");
    }
    return INT4VH_OK;
}

} // extern "C"
