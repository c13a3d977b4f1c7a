// mxfp4.hip -- rows in microscaled 4-bit floating point, and the linear layer
// between two matrices in that format, for MI355X (gfx950); formulas and order
// of rounding in int4vh_mxfp4.h.
//
// The products run on v_mfma_scale_f32_16x16x128_f8f6f4 with both operands in
// 4 bits: a lane holds 32 channels of one row, 16 bytes as they lie in memory,
// and their scale, a byte that the instruction picks out of a register.  So a
// 16-byte chunk of codes is an operand without any work on it, and LDS moves
// what the codes take in memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>
#include <type_traits>

#include "int4vh.h"
#include "int4vh_internal.h"
#include "int4vh_mxfp4.h"
#include "linear_common.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace {

using namespace int4vh_detail;

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct __attribute__((packed, aligned(1))) Words1 { uint32_t w[4]; };

constexpr int kMaxK = 65536;

// ---------------------------------------------------------------- quantisation

// 8 consecutive values, as binary32.
template <int kDtype>
__device__ __forceinline__ void load_values8(const void *p, float (&v)[8])
{
    if constexpr (kDtype == INT4VH_ROWS_F32) {
        const Words4 a = static_cast<const Words4 *>(p)[0], b = static_cast<const Words4 *>(p)[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(a.w[j]);
            v[4 + j] = __uint_as_float(b.w[j]);
        }
    } else {
        const Words2 a = *static_cast<const Words2 *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = from_bits16((a.w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, kDtype);
    }
}

template <int kDtype>
__device__ __forceinline__ void store_values8(void *p, const float (&v)[8])
{
    if constexpr (kDtype == INT4VH_ROWS_F32) {
        Words4 a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a.w[j] = __float_as_uint(v[j]);
            b.w[j] = __float_as_uint(v[4 + j]);
        }
        static_cast<Words4 *>(p)[0] = a;
        static_cast<Words4 *>(p)[1] = b;
    } else {
        Words2 a;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a.w[j] = to_bits16(v[2 * j], kDtype) | (to_bits16(v[2 * j + 1], kDtype) << 16);
        *static_cast<Words2 *>(p) = a;
    }
}

// 8 channels per thread: 4 neighbouring lanes hold the 32 that share a scale.
// Grid (chunks of 8 of a row, rows), or the whole matrix as one row.
template <int kDtype>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(const void *x, long long x_stride, int M, long long chunks,
                                                             uint32_t *codes, uint8_t *scales)
{
    constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;
    const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
    if (c >= chunks)                           // chunks is a multiple of 4: lanes leave by fours
        return;
    for (int m = blockIdx.y; m < M; m += gridDim.y) {
        float v[8];
        load_values8<kDtype>(static_cast<const char *>(x) + ((size_t)m * x_stride + 8 * c) * kSize, v);
        uint32_t peak = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = __float_as_uint(v[j]) & 0x7FFFFFFFu;
            peak = w > peak ? w : peak;
        }
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
            const uint32_t o = __shfl_xor(peak, off);
            peak = o > peak ? o : peak;
        }
        // the exponent of the largest value less 2, that of the largest code
        const int e = (int)(peak >> 23);
        const int s = e == 255 ? 255 : max(e - 2, 0);
        uint32_t q = 0u;
        if (s < 255) {
            // scaled exactly (what becomes subnormal is far below half the smallest code)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_amdgcn_ldexpf(v[j], 127 - s);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], 1.0f, 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], 1.0f, 1);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], 1.0f, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], 1.0f, 3);
        }
        codes[(size_t)m * chunks + c] = q;
        if ((threadIdx.x & 3) == 0)
            scales[((size_t)m * chunks + c) >> 2] = (uint8_t)s;
    }
}

template <int kDtype>
__global__ void __launch_bounds__(256) dequantize_mxfp4_kernel(const uint32_t *codes, const uint8_t *scales,
                                                               long long chunks, void *out)
{
    constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;
    const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
    if (c >= chunks)
        return;
    const uint32_t q = codes[c];
    const int s = scales[c >> 2];
    f32x2 p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = s == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(p[j >> 1][j & 1], s - 127);
    store_values8<kDtype>(static_cast<char *>(out) + (size_t)c * 8 * kSize, v);
}

// ---------------------------------------------------------------- products

struct MxArgs {
    const uint8_t *x, *x_scales;   // [M, K/2], [M, K/32]
    const uint8_t *w, *w_scales;   // [N, K/2], [N, K/32]
    const void *bias;              // [N] of dtype, or null
    const void *residual;          // rows residual_stride apart, or null
    long long residual_stride;
    void *out;                     // rows out_stride apart
    long long out_stride;
    float *parts;                  // [splits, M, n_pad] partial sums, or null
    int M, N, K;
    int n_pad;                     // N rounded up to 4
    int activation, dtype;
    int splits, split_steps;       // parts of K, and steps of 128 channels in each
    int tiles_m, tiles_n;
};

// The product of 16 weight rows and 16 activation rows over 128 channels; the
// scales are byte kByte of their registers.
template <int kByte>
__device__ __forceinline__ f32x4 mma(const u32x4 &w, const u32x4 &x, const f32x4 &acc, uint32_t ws, uint32_t xs)
{
    const i32x8 A = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 B = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc, 4, 4, kByte, (int)ws, kByte, (int)xs);
}

__device__ __forceinline__ float column_bias(const MxArgs &a, int n)
{
    return a.bias ? load_one(a.bias, n, a.dtype) : 0.0f;
}

__device__ __forceinline__ void finish_one(const MxArgs &a, int m, int n, float acc, float bias)
{
    float y[1] = {acc + bias};
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
__device__ __forceinline__ void finish_four(const MxArgs &a, int m, int n, const f32x4 &acc, const float (&bias)[4],
                                            bool with, uint2 res)
{
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        y[r] = acc[r] + bias[r];
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

// ---------------------------------------------------------------- up to 16 rows
constexpr int kSWaves = 8;
constexpr int kSThreads = 64 * kSWaves;
constexpr int kSMaxSteps = 8;                         // steps of 128 channels per wave
constexpr int kSMaxK = kSWaves * kSMaxSteps * 128;    // 8192 channels per workgroup

// Grid (workgroups over tiles of 16 weight rows, parts of K); kSteps: steps per
// wave, whose activations stay in registers.  The waves' sums meet in LDS, and
// are added in the order of the waves.
template <int kSteps>
__global__ void __launch_bounds__(kSThreads) mx_stream_kernel(MxArgs a)
{
    __shared__ __attribute__((aligned(16))) float s_part[2][kSWaves][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n16 = lane & 15, grp = lane >> 4;
    const int blocks = a.K / 32;
    const int c_begin = (int)blockIdx.y * a.split_steps * 4, c_end = min(blocks, c_begin + a.split_steps * 4);
    const int c0 = c_begin + wave * (kSteps * 4) + grp;         // this lane's first block of 32 channels

    auto load_w = [&](int tile, u32x4 (&q)[kSteps], uint32_t (&s)[kSteps]) {
        const size_t row = min(tile * 16 + n16, a.N - 1);
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int c = min(c0 + 4 * u, blocks - 1);          // past the end: it meets zero codes
            q[u] = *reinterpret_cast<const u32x4 *>(a.w + (row * blocks + c) * 16);
            s[u] = a.w_scales[row * blocks + c];
        }
    };
    u32x4 q[kSteps];
    uint32_t s[kSteps];
    int tile = blockIdx.x;
    load_w(tile, q, s);
    u32x4 x[kSteps];
    uint32_t xs[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int c = c0 + 4 * u;
        x[u] = u32x4{0, 0, 0, 0};
        xs[u] = 127u;
        if (n16 < a.M && c < c_end) {
            x[u] = *reinterpret_cast<const u32x4 *>(a.x + ((size_t)n16 * blocks + c) * 16);
            xs[u] = a.x_scales[(size_t)n16 * blocks + c];
        }
    }
    const int m = tid >> 4, nn = tid & 15;             // the output element of this thread in every tile
    for (int buf = 0; tile < a.tiles_n; buf ^= 1) {
        const int next = tile + gridDim.x, n = tile * 16 + nn;
        const float bs = column_bias(a, min(n, a.N - 1));
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
            acc = mma<0>(q[u], x[u], acc, s[u], xs[u]);
        if (next < a.tiles_n)
            load_w(next, q, s);
        // D: column = activation row lane & 15, rows = weight rows 4 * grp + r
        *reinterpret_cast<f32x4 *>(&s_part[buf][wave][lane * 4]) = acc;
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        barrier_no_fence();                            // the other buffer is the next tile's
        if (m < a.M && n < a.N) {
            const int at = ((nn >> 2) * 16 + m) * 4 + (nn & 3);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kSWaves; ++w)
                sum += s_part[buf][w][at];
            if (a.parts)
                a.parts[((size_t)blockIdx.y * a.M + m) * a.n_pad + n] = sum;
            else
                finish_one(a, m, n, sum, bs);
        }
        tile = next;
    }
}

// ---------------------------------------------------------------- tiles
// A workgroup computes kWM*kMB*16 activation rows x kWN*kNB*16 weight rows
// with kWM x kWN waves.  Per step of 128 channels each thread brings 16-byte
// chunks through registers into LDS, kDepth steps ahead (two LDS buffers, one
// barrier a step); 4 consecutive lanes load a row's 64 bytes.  LDS holds blocks
// of 16 rows: chunk c of row r lies in slot 4 r + (c ^ (r / 4 % 4)), which
// spreads both the writes (lanes along a row) and the reads (lanes along a
// column) over the banks.  The scales go by spans of 4 steps: a thread brings a
// row's 16 bytes and writes them so that a lane reads its own four steps' as
// one register.
template <int kWM, int kWN, int kMB, int kNB, int kDepth, bool kWhole>
__global__ void __launch_bounds__(64 * kWM *kWN) mx_tile_kernel(MxArgs a)
{
    constexpr int kThreads = 64 * kWM * kWN;
    constexpr int kBM = kWM * kMB, kBN = kWN * kNB;           // blocks of 16
    constexpr int kAPer = kBM * 64 / kThreads, kWPer = kBN * 64 / kThreads;
    static_assert(kAPer * kThreads == kBM * 64 && kWPer * kThreads == kBN * 64, "whole chunks per thread");
    static_assert(4 % kDepth == 0, "registers repeat with the spans");
    constexpr int kRows = (kBM + kBN) * 16, kSPer = (kRows + kThreads - 1) / kThreads;
    struct Lds {
        u32x4 x[kBM][64];
        u32x4 w[kBN][64];
    };
    struct Mem {
        Lds step[2];
        u32x4 scale[2][kRows];
    };
    // the epilogue's use of LDS (per wave: 16 rows of sums)
    constexpr int kCols = kNB * 16, kPitch = kCols + 4;        // the pitch spreads the rows over the banks
    constexpr int kArea = 16 * kPitch;
    constexpr size_t kTurn = 4 * kWM * kWN * kArea;
    __shared__ __attribute__((aligned(16))) uint8_t mem[sizeof(Mem) > kTurn ? sizeof(Mem) : kTurn];
    Mem &lds = *reinterpret_cast<Mem *>(mem);
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
    const int blocks = a.K / 32;
    const int s0 = part * a.split_steps, s1 = min(s0 + a.split_steps, (blocks + 3) / 4);

    // Rows past the end load the last one (never stored).  Addresses are a
    // uniform base, advanced by the step, and a 32-bit offset per chunk.
    const int cc = tid & 3;                                    // this thread's chunk of its rows
    const uint8_t *xbase = a.x + (size_t)m0 * blocks * 16, *wbase = a.w + (size_t)n0 * blocks * 16;
    uint32_t xoff[kAPer], woff[kWPer];
    const int r0 = tid >> 2, slot = (r0 >> 4) * 64 + (r0 & 15) * 4 + (cc ^ ((r0 >> 2) & 3));
#pragma unroll
    for (int j = 0; j < kAPer; ++j)
        xoff[j] = (uint32_t)(min(r0 + j * (kThreads / 4), a.M - 1 - m0) * blocks + cc) * 16u;
#pragma unroll
    for (int j = 0; j < kWPer; ++j)
        woff[j] = (uint32_t)(min(r0 + j * (kThreads / 4), a.N - 1 - n0) * blocks + cc) * 16u;
    // Loads past the last step repeat it, and chunks past K load the row's last
    // one, so that every step issues the same loads without a branch; the
    // activations' codes past K are cleared on their way to LDS.
    u32x4 rx[kDepth][kAPer], rw[kDepth][kWPer];
    auto load = [&](int d, int step) {
        const int s = min(step, s1 - 1);
        const uint8_t *px = xbase + (size_t)s * 64, *pw = wbase + (size_t)s * 64;
        const uint32_t back = kWhole ? 0u : 16u * (uint32_t)max(0, s * 4 + cc - (blocks - 1));
#pragma unroll
        for (int j = 0; j < kAPer; ++j)
            rx[d][j] = *reinterpret_cast<const u32x4 *>(px + (xoff[j] - back));
#pragma unroll
        for (int j = 0; j < kWPer; ++j)
            rw[d][j] = *reinterpret_cast<const u32x4 *>(pw + (woff[j] - back));
    };
    auto store = [&](int d, int s, Lds &l) {
        if (!kWhole) {
            const bool live = s * 4 + cc < blocks;
#pragma unroll
            for (int j = 0; j < kAPer; ++j)
                rx[d][j] = live ? rx[d][j] : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < kAPer; ++j)
            (&l.x[0][0])[slot + j * kThreads] = rx[d][j];
#pragma unroll
        for (int j = 0; j < kWPer; ++j)
            (&l.w[0][0])[slot + j * kThreads] = rw[d][j];
    };
    // a thread's rows of scales: activations, then weights
    const uint8_t *srow[kSPer];
#pragma unroll
    for (int j = 0; j < kSPer; ++j) {
        const int r = min(tid + j * kThreads, kRows - 1);
        srow[j] = r < kBM * 16 ? a.x_scales + (size_t)min(m0 + r, a.M - 1) * blocks
                               : a.w_scales + (size_t)min(n0 + r - kBM * 16, a.N - 1) * blocks;
    }
    uint32_t rs[kSPer][4];
    auto load_scales = [&](int step) {                         // of steps step .. step + 3
        const int s = min(step, (s1 - 1) & ~3);
#pragma unroll
        for (int j = 0; j < kSPer; ++j) {
            if (kWhole) {
                const Words1 v = *reinterpret_cast<const Words1 *>(srow[j] + 4 * s);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rs[j][i] = v.w[i];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    rs[j][i] = 0u;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int c = 4 * s + 4 * i + b;
                        const uint32_t v = srow[j][min(c, blocks - 1)];
                        rs[j][i] |= (c < blocks ? v : 0u) << (8 * b);
                    }
                }
            }
        }
    };
    auto store_scales = [&](u32x4 *to) {
#pragma unroll
        for (int j = 0; j < kSPer; ++j) {
            const uint32_t lo = __builtin_amdgcn_perm(rs[j][1], rs[j][0], 0x05010400u);
            const uint32_t hi = __builtin_amdgcn_perm(rs[j][1], rs[j][0], 0x07030602u);
            const uint32_t lo2 = __builtin_amdgcn_perm(rs[j][3], rs[j][2], 0x05010400u);
            const uint32_t hi2 = __builtin_amdgcn_perm(rs[j][3], rs[j][2], 0x07030602u);
            if (kRows % kThreads == 0 || tid + j * kThreads < kRows)
                to[tid + j * kThreads] = u32x4{__builtin_amdgcn_perm(lo2, lo, 0x05040100u),
                                               __builtin_amdgcn_perm(lo2, lo, 0x07060302u),
                                               __builtin_amdgcn_perm(hi2, hi, 0x05040100u),
                                               __builtin_amdgcn_perm(hi2, hi, 0x07060302u)};
        }
    };

    f32x4 acc[kMB][kNB];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};

    load_scales(s0);
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        load(d, s0 + d);
    store_scales(lds.scale[0]);
    store(0, s0, lds.step[0]);
    const int rslot = n16 * 4 + (grp ^ ((n16 >> 2) & 3));
    uint32_t xs[kMB], ws[kNB];
    auto step = [&](const Lds &l, auto byte) {
        u32x4 x[kMB];
#pragma unroll
        for (int i = 0; i < kMB; ++i)
            x[i] = l.x[wm * kMB + i][rslot];
#pragma unroll
        for (int j = 0; j < kNB; ++j) {
            const u32x4 w = l.w[wn * kNB + j][rslot];
#pragma unroll
            for (int i = 0; i < kMB; ++i)
                acc[i][j] = mma<decltype(byte)::value>(w, x[i], acc[i][j], ws[j], xs[i]);
        }
    };
    auto turn_step = [&](int s, int sbuf, auto byte) {
        constexpr int i = decltype(byte)::value;
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        barrier_no_fence();
        if constexpr (i == 0) {
            const uint32_t *sc = reinterpret_cast<const uint32_t *>(lds.scale[sbuf]);
#pragma unroll
            for (int k = 0; k < kMB; ++k)
                xs[k] = sc[(wm * kMB + k) * 64 + lane / 16 + n16 * 4];
#pragma unroll
            for (int k = 0; k < kNB; ++k)
                ws[k] = sc[(kBM + wn * kNB + k) * 64 + lane / 16 + n16 * 4];
            load_scales(s + 4);
        }
        load(i % kDepth, s + i + kDepth);
        step(lds.step[i & 1], byte);
        store((i + 1) % kDepth, s + i + 1, lds.step[(i + 1) & 1]);
        if constexpr (i == 3)
            store_scales(lds.scale[sbuf ^ 1]);
    };
    // whole spans: steps past K multiply zeros (a way out of the middle of a span
    // would copy all sums)
    int sbuf = 0;
    for (int s = s0; s < s1; s += 4, sbuf ^= 1) {
        turn_step(s, sbuf, std::integral_constant<int, 0>());
        turn_step(s, sbuf, std::integral_constant<int, 1>());
        turn_step(s, sbuf, std::integral_constant<int, 2>());
        turn_step(s, sbuf, std::integral_constant<int, 3>());
    }

    // D: column = activation row lane & 15, rows = weight rows 4 * grp + r.
    // Each wave turns its sums around in LDS, 16 activation rows at a time, so
    // that its lanes hold four columns of a row and rows are written whole.
    // The residual of the next 16 rows is asked for before these are stored: a
    // wait for a load also waits for the stores in front of it.
    float *turn = reinterpret_cast<float *>(mem) + wave * kArea;
    constexpr int kLanes = kCols / 4, kStep = 64 / kLanes, kIter = 16 / kStep;   // lanes of a row; rows at a time
    const int c4 = (lane % kLanes) * 4, n = n0 + wn * kCols + c4, lr = lane / kLanes;
    const int mw = m0 + wm * kMB * 16;
    float bs[4];
    Pair2 res[2][kIter];
    // The usual case handles four columns at a time, with a 16-bit residual or
    // none; rows that end inside a lane's four columns, and binary32 residuals,
    // go element by element.
    const bool wide = !a.parts && a.N % 4 == 0 && (!a.residual || a.dtype != INT4VH_ROWS_F32);
    const bool early = wide && a.residual;
    auto load_residual = [&](int i) {
#pragma unroll
        for (int k = 0; k < kIter; ++k) {
            const int m = min(mw + i * 16 + lr + k * kStep, a.M - 1);
            res[i & 1][k] = *reinterpret_cast<const Pair2 *>(static_cast<const uint16_t *>(a.residual) +
                                                             (size_t)m * a.residual_stride + min(n, a.N - 4));
        }
    };
    if (!a.parts) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            bs[r] = column_bias(a, min(n + r, a.N - 1));
        if (early)
            load_residual(0);
    }
    __builtin_amdgcn_s_waitcnt(0);
    barrier_no_fence();                                        // the last step's reads are done
#pragma unroll
    for (int i = 0; i < kMB; ++i) {
        const int mi = mw + i * 16;
#pragma unroll
        for (int j = 0; j < kNB; ++j)
            *reinterpret_cast<f32x4 *>(turn + n16 * kPitch + j * 16 + 4 * grp) = acc[i][j];
        if (early && i + 1 < kMB)
            load_residual(i + 1);
        wave_fence();
        if (wide) {
#pragma unroll
            for (int k = 0; k < kIter; ++k) {
                const int r = lr + k * kStep;
                const f32x4 v = *reinterpret_cast<const f32x4 *>(turn + r * kPitch + c4);
                if (mi + r < a.M && n < a.N)
                    finish_four(a, mi + r, n, v, bs, early, make_uint2(res[i & 1][k].w[0], res[i & 1][k].w[1]));
            }
        } else if (a.parts) {
#pragma nounroll
            for (int r = lr; r < 16; r += kStep)
                if (mi + r < a.M && n < a.N)
                    *reinterpret_cast<f32x4 *>(&a.parts[((size_t)part * a.M + mi + r) * a.n_pad + n]) =
                        *reinterpret_cast<const f32x4 *>(turn + r * kPitch + c4);
        } else {
#pragma nounroll
            for (int e = lane; e < 16 * kCols; e += 64) {
                const int m = mi + e / kCols, c = n0 + wn * kCols + e % kCols;
                if (m < a.M && c < a.N)
                    finish_one(a, m, c, turn[e / kCols * kPitch + e % kCols], column_bias(a, c));
            }
        }
        wave_fence();
    }
}

// The parts' sums, in their order, and the epilogue: one thread per element.
__global__ void __launch_bounds__(256) mx_join_kernel(MxArgs a)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)a.M * a.N)
        return;
    const int m = (int)(i / a.N), n = (int)(i % a.N);
    float sum = 0.0f;
    for (int p = 0; p < a.splits; ++p)
        sum += a.parts[((size_t)p * a.M + m) * a.n_pad + n];
    finish_one(a, m, n, sum, column_bias(a, n));
}

// ---------------------------------------------------------------- host side

enum Kind { kStream, kTile32, kTile128 };
struct Plan {
    Kind kind;
    int splits, split_steps;
    int tiles_m, tiles_n;
};

long long tiles_of(int M, int N, int bm, int bn)
{
    return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

Plan plan_for(int M, int N, int K, int cus)
{
    Plan p;
    const int steps = (K + 127) / 128;
    p.splits = 1;
    if (M <= 16) {
        p.kind = kStream;
        p.tiles_m = 1;
        p.tiles_n = (N + 15) / 16;
        p.splits = (K + kSMaxK - 1) / kSMaxK;
    } else {
        p.kind = 2 * tiles_of(M, N, 128, 128) >= cus ? kTile128 : kTile32;
        const int bm = p.kind == kTile128 ? 128 : 32;
        p.tiles_m = (M + bm - 1) / bm;
        p.tiles_n = (N + 127) / 128;
        // few tiles: parts of at least 4 steps, up to two workgroups a compute unit
        if (p.kind == kTile32)
            while (2 * p.splits * tiles_of(M, N, 32, 128) <= 2ll * cus && steps / (2 * p.splits) >= 4)
                p.splits *= 2;
    }
    p.split_steps = (steps + p.splits - 1) / p.splits;
    if (p.splits > 1)                          // whole spans of scales
        p.split_steps = (p.split_steps + 3) / 4 * 4;
    p.splits = (steps + p.split_steps - 1) / p.split_steps;
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
    return K <= kMaxK && N <= (1 << 24) && M <= (1 << 20) && (long long)M * N < (1ll << 40);
}

void launch_stream(const MxArgs &a, dim3 grid, hipStream_t s)
{
    const int per_wave = (a.split_steps + kSWaves - 1) / kSWaves;
    const dim3 block(kSThreads);
    if (per_wave <= 1)
        hipLaunchKernelGGL(mx_stream_kernel<1>, grid, block, 0, s, a);
    else if (per_wave <= 2)
        hipLaunchKernelGGL(mx_stream_kernel<2>, grid, block, 0, s, a);
    else if (per_wave <= 3)
        hipLaunchKernelGGL(mx_stream_kernel<3>, grid, block, 0, s, a);
    else if (per_wave <= 5)
        hipLaunchKernelGGL(mx_stream_kernel<5>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(mx_stream_kernel<8>, grid, block, 0, s, a);
}

template <int kWM, int kWN, int kMB, int kNB, int kDepth>
void launch_tiles(const MxArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((long long)a.tiles_m * a.tiles_n * a.splits)), block(64 * kWM * kWN);
    if (a.K % 512 == 0)
        hipLaunchKernelGGL((mx_tile_kernel<kWM, kWN, kMB, kNB, kDepth, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((mx_tile_kernel<kWM, kWN, kMB, kNB, kDepth, false>), grid, block, 0, s, a);
}

template <int kDtype>
void launch_quantize(const void *x, int64_t x_stride, int M, int H, uint8_t *codes, uint8_t *scales, hipStream_t s)
{
    const bool flat = M == 1 || x_stride == H;         // one long row
    const long long chunks = flat ? (long long)M * H / 8 : H / 8;
    const int rows = flat ? 1 : M;
    const dim3 grid((unsigned)((chunks + 255) / 256), rows < 65535 ? rows : 65535);
    hipLaunchKernelGGL(quantize_mxfp4_kernel<kDtype>, grid, dim3(256), 0, s, x, (long long)x_stride, rows, chunks,
                       reinterpret_cast<uint32_t *>(codes), scales);
}

template <int kDtype>
void launch_dequantize(const uint8_t *codes, const uint8_t *scales, int M, int H, void *out, hipStream_t s)
{
    const long long chunks = (long long)M * H / 8;
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<kDtype>, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, s,
                       reinterpret_cast<const uint32_t *>(codes), scales, chunks, out);
}

} // namespace

extern "C" {

int quantize_rows_mxfp4(const void *x, int64_t x_stride, int dtype, int M, int H, uint8_t *codes, uint8_t *scales,
                        void *stream)
{
    if (M < 1 || H < 32 || H % 32 || !rows_known(dtype) || !x || !codes || !scales || (M > 1 && x_stride < H))
        return INT4VH_EINVAL;
    if (!rows_aligned(x, rows_size(dtype)) || !rows_aligned(codes, 4))
        return INT4VH_EALIGN;
    if (H > kMaxK || (long long)M * H >= (1ll << 40))
        return INT4VH_EUNSUPPORTED;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == INT4VH_ROWS_F16)
        launch_quantize<INT4VH_ROWS_F16>(x, x_stride, M, H, codes, scales, s);
    else if (dtype == INT4VH_ROWS_BF16)
        launch_quantize<INT4VH_ROWS_BF16>(x, x_stride, M, H, codes, scales, s);
    else
        launch_quantize<INT4VH_ROWS_F32>(x, x_stride, M, H, codes, scales, s);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? INT4VH_OK : hip_fail(e, "mxfp4 quantisation kernel launch");
}

int dequantize_rows_mxfp4(const uint8_t *codes, const uint8_t *scales, int M, int H, void *out, int dtype,
                          void *stream)
{
    if (M < 1 || H < 32 || H % 32 || !rows_known(dtype) || !codes || !scales || !out)
        return INT4VH_EINVAL;
    if (!rows_aligned(codes, 16) || !rows_aligned(out, rows_size(dtype)))
        return INT4VH_EALIGN;
    if (H > kMaxK || (long long)M * H >= (1ll << 40))
        return INT4VH_EUNSUPPORTED;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == INT4VH_ROWS_F16)
        launch_dequantize<INT4VH_ROWS_F16>(codes, scales, M, H, out, s);
    else if (dtype == INT4VH_ROWS_BF16)
        launch_dequantize<INT4VH_ROWS_BF16>(codes, scales, M, H, out, s);
    else
        launch_dequantize<INT4VH_ROWS_F32>(codes, scales, M, H, out, s);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? INT4VH_OK : hip_fail(e, "mxfp4 dequantisation kernel launch");
}

size_t linear_mxfp4_rows_workspace_bytes(int M, int N, int K)
{
    if (!sizes_ok(M, N, K) || !sizes_supported(M, N, K))
        return 0;
    return parts_bytes(plan_for(M, N, K, current_cus()), M, N);
}

int linear_mxfp4_rows(const uint8_t *codes, const uint8_t *scales, const uint8_t *w_codes, const uint8_t *w_scales,
                      const void *bias, int activation, const void *residual, int64_t residual_stride, int M, int N,
                      int K, void *out, int64_t out_stride, int dtype, void *workspace, size_t workspace_bytes,
                      void *stream)
{
    if (!sizes_ok(M, N, K) || !codes || !scales || !w_codes || !w_scales || !out || !rows_known(dtype) ||
        activation < INT4VH_ACT_NONE || activation > INT4VH_ACT_SILU)
        return INT4VH_EINVAL;
    if (M > 1 && (out_stride < N || (residual && residual_stride < N)))
        return INT4VH_EINVAL;
    const size_t el = rows_size(dtype);
    if (!rows_aligned(codes, 16) || !rows_aligned(w_codes, 16) || !rows_aligned(bias, el) ||
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
    MxArgs a;
    a.x = codes;
    a.x_scales = scales;
    a.w = w_codes;
    a.w_scales = w_scales;
    a.bias = bias;
    a.residual = residual;
    a.residual_stride = residual_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.parts = need ? static_cast<float *>(workspace) : nullptr;
    a.M = M;
    a.N = N;
    a.K = K;
    a.n_pad = (N + 3) / 4 * 4;
    a.activation = activation;
    a.dtype = dtype;
    a.splits = p.splits;
    a.split_steps = p.split_steps;
    a.tiles_m = p.tiles_m;
    a.tiles_n = p.tiles_n;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.kind == kStream)
        launch_stream(a, dim3(p.tiles_n < 2 * cus ? p.tiles_n : 2 * cus, p.splits), s);
    else if (p.kind == kTile32)
        launch_tiles<1, 2, 2, 4, 2>(a, s);
    else
        launch_tiles<2, 2, 4, 4, 2>(a, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return hip_fail(e, "mxfp4 linear kernel launch");
    if (need) {
        const long long n1 = (long long)M * N;
        hipLaunchKernelGGL(mx_join_kernel, dim3((unsigned)((n1 + 255) / 256)), dim3(256), 0, s, a);
        e = hipGetLastError();
        if (e != hipSuccess)
            return hip_fail(e, "mxfp4 join kernel launch");
    }
    return INT4VH_OK;
}

} // extern "C"
