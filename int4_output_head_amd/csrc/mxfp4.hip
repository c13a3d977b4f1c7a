// mxfp4.hip -- rows in microscaled 4-bit floating point, and the linear layer
// between two matrices in that format, for MI355X (gfx950); formulas and order
// of rounding in int4vh_mxfp4.h.
//
// The products run on v_mfma_scale_f32_16x16x128 and _32x32x64_f8f6f4 with both
// operands in 4 bits: a lane holds 32 channels of one row, 16 bytes as they lie in
// memory, and their scale, a byte that the instruction picks out of a register.
// So a 16-byte chunk of codes is an operand without any work on it, and LDS moves
// what the codes take in memory.  The larger form reaches 8.0 PFLOP/s on this
// card in a loop of its own, the smaller one 5.9.
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
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct __attribute__((packed, aligned(1))) Word1 { uint32_t w; };
struct __attribute__((packed, aligned(1))) Words1 { uint32_t w[4]; };
typedef unsigned long long u64;

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
// Grid (chunks of 8 of a row, rows), or the whole matrix as one row.  Bound by
// memory: 4096 x 8192 in bfloat16, 85 MB, takes 17.6 us (4.8 TB/s), and the way
// back below 13.8.
template <int kDtype>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(const void *x, long long x_stride, int M, long long chunks,
                                                             uint32_t *codes, uint8_t *scales)
{
    constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;
    const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
    if (c >= chunks)                           // chunks is a multiple of 4: lanes leave by fours
        return;
    // (unsigned: a step past the last of 2^31 - 1 rows passes 31 bits)
    for (unsigned m = blockIdx.y; m < (unsigned)M; m += gridDim.y) {
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
    for (long long c = (long long)blockIdx.x * 256 + threadIdx.x; c < chunks; c += (long long)gridDim.x * 256) {
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
    int splits, split_spans;       // parts of K, and spans of 512 channels in each
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

// 32 weight rows and 32 activation rows over 64 channels; the scales are byte
// kByte of their registers.
template <int kByte>
__device__ __forceinline__ f32x16 mma32(const u32x4 &w, const u32x4 &x, const f32x16 &acc, uint32_t ws, uint32_t xs)
{
    const i32x8 A = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 B = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, acc, 4, 4, kByte, (int)ws, kByte, (int)xs);
}

__device__ __forceinline__ float column_bias(const MxArgs &a, int n)
{
    return a.bias ? load_one(a.bias, n, a.dtype) : 0.0f;
}

// Four consecutive output elements at `to`, but for the residual, whose 16-bit words
// res are added where `with` is set.
template <int kDtype>
__device__ __forceinline__ void store_four(void *to, const f32x4 &y, bool with, uint2 res)
{
    if constexpr (kDtype == INT4VH_ROWS_F32) {
        Words4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v.w[r] = __float_as_uint(y[r]);
        *static_cast<Words4 *>(to) = v;
    } else {
        f32x4 z = y;
        if (with) {
            z[0] += from_bits16(res.x & 0xFFFFu, kDtype);
            z[1] += from_bits16(res.x >> 16, kDtype);
            z[2] += from_bits16(res.y & 0xFFFFu, kDtype);
            z[3] += from_bits16(res.y >> 16, kDtype);
        }
        Pair2 v;
        v.w[0] = to_bits16(z[0], kDtype) | (to_bits16(z[1], kDtype) << 16);
        v.w[1] = to_bits16(z[2], kDtype) | (to_bits16(z[3], kDtype) << 16);
        *static_cast<Pair2 *>(to) = v;
    }
}

// One output element, but for the residual.
__device__ __forceinline__ void store_one(const MxArgs &a, int m, int n, float y)
{
    if (a.residual)
        y += load_one(a.residual, (size_t)m * a.residual_stride + n, a.dtype);
    const size_t o = (size_t)m * a.out_stride + n;
    if (a.dtype == INT4VH_ROWS_F32)
        static_cast<float *>(a.out)[o] = y;
    else
        static_cast<uint16_t *>(a.out)[o] = (uint16_t)to_bits16(y, a.dtype);
}

__device__ __forceinline__ void finish_one(const MxArgs &a, int m, int n, float acc, float bias)
{
    float y[1] = {acc + bias};
    activate(y, a.activation);
    store_one(a, m, n, y[0]);
}

// ---------------------------------------------------------------- up to 16 rows
constexpr int kSWaves = 8;
constexpr int kSThreads = 64 * kSWaves;
constexpr int kSMaxSteps = 8;                         // steps of 128 channels per wave
constexpr int kSMaxK = kSWaves * kSMaxSteps * 128;    // 8192 channels per workgroup

// Grid (workgroups over tiles of 16 weight rows, parts of K); kSteps: steps per
// wave, whose activations stay in registers.  The waves' sums meet in LDS, and
// are added in the order of the waves.  Scales: a lane needs a byte of each step,
// the one of its own 32 channels; a row's 4 bytes of a step are loaded as a word
// by one lane, step u's by the lanes of group u % 4, and passed on (kWhole: K is
// a multiple of 128; otherwise each lane loads its bytes).  Bound by the weights'
// stream where there are enough (16 x 34816 x 5120: 19.4 us, 4.9 TB/s), and by
// latencies where there are not (16 x 5120 x 5120: 7 us, 320 tiles for 512
// workgroups).
template <int kSteps, bool kWhole>
__global__ void __launch_bounds__(kSThreads, kSteps > 6 ? 2 : 4) mx_stream_kernel(MxArgs a)
{
    // the pitch spreads 16 rows' chunks over the banks
    constexpr int kRow = 4 * kSteps, kPitch = kRow + (kSteps % 2 ? 0 : 4);
    __shared__ __attribute__((aligned(16))) float s_part[2][kSWaves][256];
    __shared__ u32x4 s_turn[kSWaves][16 * kPitch];
    constexpr int kWords = kWhole ? (kSteps + 3) / 4 : kSteps;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, grp = lane >> 4;
    const int blocks = a.K / 32;
    const int c_begin = (int)blockIdx.y * a.split_spans * 16, c_end = min(blocks, c_begin + a.split_spans * 16);
    const int c0 = c_begin + wave * (kSteps * 4);               // this wave's first block of 32 channels

    // Sixteen rows' codes, 64 chunks an instruction along the rows (16 rows' 64 bytes
    // each an instruction meet in few sets of L1 where rows are a multiple of 512
    // bytes apart: 16 x 5120 x 5120 took 9.0 us instead of 7.0).  Rows and chunks past
    // the end are any valid ones, which meet zero codes.
    auto load_codes = [&](const uint8_t *codes, int last, u32x4 (&q)[kSteps]) {
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int i = 64 * u + lane, r = min(i / kRow, last), c = min(c0 + i % kRow, blocks - 1);
            q[u] = *reinterpret_cast<const u32x4 *>(codes + ((uint32_t)r * (uint32_t)blocks + (uint32_t)c) * 16u);
        }
    };
    // To the products' layout, in LDS of the wave's own.
    auto turn = [&](const u32x4 (&q)[kSteps]) {
        wave_fence();
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int i = 64 * u + lane;
            s_turn[wave][i / kRow * kPitch + i % kRow] = q[u];
        }
        wave_fence();
    };
    auto turned = [&](int u) { return s_turn[wave][n16 * kPitch + 4 * u + grp]; };
    auto load_words = [&](const uint8_t *scales, int r, uint32_t (&s)[kWords]) {
        const uint8_t *row = scales + (uint32_t)r * (uint32_t)blocks;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (kWhole) {
                const Word1 v = *reinterpret_cast<const Word1 *>(row + min(c0 + 16 * i + 4 * grp, blocks - 4));
                s[i] = v.w;
            } else {
                s[i] = row[min(c0 + 4 * i + grp, blocks - 1)];
            }
        }
    };
    // step u's scale, in the lowest byte
    auto scale = [&](const uint32_t (&s)[kWords], int u) {
        if constexpr (kWhole)
            return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * ((u & 3) * 16 + n16), (int)s[u >> 2]) >> (8 * grp);
        else
            return s[u];
    };
    auto load_w = [&](int tile, u32x4 (&q)[kSteps], uint32_t (&s)[kWords]) {
        const int last = a.N - 1 - tile * 16;
        load_codes(a.w + (size_t)tile * 16 * blocks * 16, last, q);
        load_words(a.w_scales + (size_t)tile * 16 * blocks, min(n16, last), s);
    };
    u32x4 q[kSteps];
    uint32_t s[kWords], xw[kWords];
    int tile = blockIdx.x;
    load_w(tile, q, s);
    u32x4 x[kSteps];
    uint32_t xs[kSteps];
    load_codes(a.x, a.M - 1, x);
    load_words(a.x_scales, min(n16, a.M - 1), xw);
    turn(x);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const bool live = n16 < a.M && c0 + 4 * u + grp < c_end;
        x[u] = live ? turned(u) : u32x4{0, 0, 0, 0};
        xs[u] = scale(xw, u);
    }
    const int m = tid >> 4, nn = tid & 15;             // the output element of this thread in every tile
    for (int buf = 0; tile < a.tiles_n; buf ^= 1) {
        const int next = tile + gridDim.x, n = tile * 16 + nn;
        const float bs = column_bias(a, min(n, a.N - 1));
        turn(q);
        uint32_t ws[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
            ws[u] = scale(s, u);
        if (next < a.tiles_n)
            load_w(next, q, s);
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
            acc = mma<0>(turned(u), x[u], acc, ws[u], xs[u]);
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
__device__ __forceinline__ uint32_t lds_at(const void *p)
{
    return (uint32_t)(size_t)(const __attribute__((address_space(3))) void *)p;
}
// Values that the compiler cannot compute with ahead of here: what follows from
// them would otherwise stay in registers all through a loop.
__device__ __forceinline__ void hold(uint32_t &a, uint32_t &b, uint32_t &c)
{
    asm volatile("" : "+v"(a), "+v"(b), "+v"(c));
}
// The lane's number, found anew.
__device__ __forceinline__ uint32_t lane_here()
{
    uint32_t lane;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(lane));
    return lane;
}
typedef const __attribute__((address_space(3))) u32x4 lds_words;
__device__ __forceinline__ lds_words *lds_pointer(uint32_t at)
{
    return (lds_words *)(size_t)at;
}
constexpr int waitcnt_vm(int n)
{
    return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8);
}

// A copy of 16 bytes per lane straight into LDS: lane l's, from base + offset,
// land at dst + 16 l.  Inline asm: the compiler would order all reads of LDS
// behind all copies that it knows to be in flight.  Nothing comes back into
// registers; the kernel waits for its copies itself.  m0 is named so that the compiler
// takes nothing of its own there for granted behind a copy (its warning is that it does
// not keep a reserved register's value across, which nobody asks for).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds16(const uint8_t *base, uint32_t offset, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(offset), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// A workgroup computes kWM*kMB*32 activation rows x kWN*kNB*32 weight rows with
// kWM x kWN waves, in steps of 256 channels.  A step's codes are copied from
// memory straight into one of kRing buffers in LDS while another is multiplied:
// 1 KB, 8 rows' 128 bytes (whole cache lines: with 64 bytes of 16 rows the
// copies alone took 187 us instead of 137 for 8192^3), an instruction.  In LDS
// chunk c of row r lies in slot 8 r + (c ^ (r / 2 % 8)), which spreads the reads
// (lanes along a column) over the banks; the copy's lanes are numbered
// accordingly.  The operands of the next quarter of a step are read while this
// one's are multiplied; the barrier stands in front of a step's last quarter, so
// that the copies into the buffer that it frees, and the reads from the other
// one, have its products to hide behind.  The scales, 16 bytes a row for 512
// channels, are copied likewise for 1024 (kWhole), or go through registers, asked
// for two steps ahead, where rows do not end with a whole span of 512 or are not
// aligned to it (1024 x 5120 x 4096: 23 us, 4128: 33; byte by byte, a step ahead, 47;
// the tiles of 128 rows spill 16 registers in this form).
//
// What bounds it is the way of the codes into LDS: without any product 8192^3
// takes 295 us of 345, without the copies 229.  128 rows and two buffers, two
// workgroups a compute unit, are the fastest where there is work for half the
// card (4096 x 5120 x 8192: 105 us; three buffers, one workgroup 144; 64 rows
// 147); a few tiles of 64 rows have a compute unit each, and there a third
// buffer hides more of memory's latency (256 x 5120 x 5120: 13.1 us, two 15.6).
template <int kWM, int kWN, int kMB, int kNB, int kRing, bool kWhole>
__global__ void __launch_bounds__(64 * kWM *kWN, kRing == 2 ? 2 : 1) mx_tile_kernel(MxArgs a)
{
    constexpr int kWaves = kWM * kWN;
    constexpr int kBM = kWM * kMB, kBN = kWN * kNB;           // blocks of 32
    constexpr int kRows = (kBM + kBN) * 32;
    constexpr int kPer = kRows / 8 / kWaves;                  // copies of a wave per step
    static_assert(kPer * kWaves * 8 == kRows && kBM * 32 % (8 * kWaves) == 0, "whole copies per wave, of one matrix each");
    struct Mem {
        u32x4 code[kRing][kRows][8];
        u32x4 scale[2][kRows][2];
    };
    // the epilogue's use of LDS (per wave: 32 rows of sums)
    constexpr int kCols = kNB * 32, kPitch = kCols + 4;        // the pitch spreads the rows over the banks
    constexpr int kArea = 32 * kPitch;
    constexpr size_t kTurn = 4 * kWaves * kArea;
    __shared__ __attribute__((aligned(16))) uint8_t mem[sizeof(Mem) > kTurn ? sizeof(Mem) : kTurn];
    Mem &lds = *reinterpret_cast<Mem *>(mem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n32 = lane & 31, half = lane >> 5;
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
    const int m0 = (first + in % rows) * kBM * 32, n0 = (in / rows) * kBN * 32;
    const int blocks = a.K / 32;
    // spans of 512 channels, two steps each
    const int p0 = part * a.split_spans, p1 = min(p0 + a.split_spans, (blocks + 15) / 16);

    // Rows past the end load the last one (never stored); copies past the last
    // step repeat it, and chunks past K are the row's last one, so that every step
    // issues the same copies without a branch.
    const int cr = wave * 8 + (lane >> 3), cc = (lane & 7) ^ ((cr >> 1) & 7);
    const uint8_t *xbase = a.x + (size_t)m0 * blocks * 16, *wbase = a.w + (size_t)n0 * blocks * 16;
    constexpr int kXPer = kBM * 32 / (8 * kWaves);             // the copies of activations
    uint32_t row = (uint32_t)cr;
    auto load = [&](int step, int buf) {
        const int s = min(step, 2 * p1 - 1);
        // (the offset added to a base is not negative)
        const uint32_t chunk = kWhole ? (uint32_t)cc : (uint32_t)min(s * 8 + cc, blocks - 1);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t r = j < kXPer ? min(row + j * 8 * kWaves, (uint32_t)(a.M - 1 - m0))
                                         : min(row + (j - kXPer) * 8 * kWaves, (uint32_t)(a.N - 1 - n0));
            copy_to_lds16((j < kXPer ? xbase : wbase) + (kWhole ? (size_t)s * 128 : 0), (r * (uint32_t)blocks + chunk) * 16u,
                          lds_at(&lds.code[buf][wave * 8 + j * 8 * kWaves][0]));
        }
    };
    // rows of scales: 32 an instruction, 32 bytes each, or one a lane through
    // registers
    const uint8_t *sxbase = a.x_scales + (size_t)m0 * blocks, *swbase = a.w_scales + (size_t)n0 * blocks;
    constexpr int kSRows = kWhole ? 32 : 64, kSCopies = kRows / kSRows, kSPer = (kSCopies + kWaves - 1) / kWaves;
    static_assert(kBM * 32 % kSRows == 0 && kRows % kSRows == 0, "a copy of scales is of one matrix");
    uint32_t sfrom[kSPer];
#pragma unroll
    for (int j = 0; j < kSPer; ++j) {
        const int r = min(wave + j * kWaves, kSCopies - 1) * kSRows + (kWhole ? lane >> 1 : lane);
        sfrom[j] = (uint32_t)(r < kBM * 32 ? min(r, a.M - 1 - m0) : min(r - kBM * 32, a.N - 1 - n0)) * (uint32_t)blocks;
    }
    auto copy_scales = [&](int span, int buf) {                // of spans `span` and the next
#pragma unroll
        for (int j = 0; j < kSPer; ++j) {
            const int b = min(wave + j * kWaves, kSCopies - 1);
            copy_to_lds16(b * kSRows < kBM * 32 ? sxbase : swbase,
                          sfrom[j] + (uint32_t)min(16 * span + 16 * (lane & 1), blocks - 16),
                          lds_at(&lds.scale[buf][b * kSRows][0]));
        }
    };
    uint32_t rs[kSPer][4];
    int skip = 0;
    auto load_scales = [&](int span) {                         // of one span
        const int s = min(span, p1 - 1);
        // the last span's are the row's last 16, less those in front of it
        const int from = min(16 * s, blocks - 16), off = 16 * s - from;
#pragma unroll
        for (int j = 0; j < kSPer; ++j) {
            const uint8_t *row = (min(wave + j * kWaves, kSCopies - 1) * kSRows < kBM * 32 ? sxbase : swbase) + sfrom[j];
            if (blocks >= 16) {
                const Words1 v = *reinterpret_cast<const Words1 *>(row + from);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rs[j][i] = v.w[i];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    rs[j][i] = 0u;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        rs[j][i] |= (4 * i + q < blocks ? (uint32_t)row[min(4 * i + q, blocks - 1)] : 0u) << (8 * q);
                }
            }
        }
        skip = blocks >= 16 ? off : 0;
    };
    auto store_scales = [&](int span) {
#pragma unroll
        for (int j = 0; j < kSPer; ++j) {
            u64 lo = (u64)rs[j][1] << 32 | rs[j][0], hi = (u64)rs[j][3] << 32 | rs[j][2];
            if (skip) {                                        // towards the first, zeros behind
                lo = skip & 8 ? hi : lo;
                hi = skip & 8 ? 0ull : hi;
                const int bits = 8 * (skip & 7);
                lo = bits ? lo >> bits | hi << (64 - bits) : lo;
                hi >>= bits;
            }
            lds.scale[(span >> 1) & 1][min(wave + j * kWaves, kSCopies - 1) * kSRows + lane][span & 1] =
                u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        }
    };

    f32x16 acc[kMB][kNB];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][j][r] = 0.0f;

    // Quarter q of a step: chunk 2 q + (lane / 32) of the lane's row.  Two sets of
    // operands take turns.
    u32x4 x[2][kMB], w[2][kNB], xs[kMB], ws[kNB];
    // addresses in LDS of the lane's first chunk; chunk c of its row lies 16 c away, bit
    // by bit
    const uint32_t turned = 16u * (uint32_t)(half ^ ((n32 >> 1) & 7));
    uint32_t ax = lds_at(&lds.code[0][wm * kMB * 32 + n32][0]) + turned;
    uint32_t aw = lds_at(&lds.code[0][(kBM + wn * kNB) * 32 + n32][0]) + turned;
    auto read = [&](int step, int buf, int q, auto tail) {
        lds_words *px = lds_pointer((ax ^ (32u * q)) + buf * (uint32_t)sizeof(lds.code[0]));
        lds_words *pw = lds_pointer((aw ^ (32u * q)) + buf * (uint32_t)sizeof(lds.code[0]));
#pragma unroll
        for (int k = 0; k < kMB; ++k)
            x[q & 1][k] = px[32 * 8 * k];
#pragma unroll
        for (int k = 0; k < kNB; ++k)
            w[q & 1][k] = pw[32 * 8 * k];
        if (!kWhole && decltype(tail)::value && step * 8 + 8 > blocks) {
            const bool live = step * 8 + 2 * q + half < blocks;
#pragma unroll
            for (int k = 0; k < kMB; ++k)
                x[q & 1][k] = live ? x[q & 1][k] : u32x4{0, 0, 0, 0};
        }
    };
    auto read_scales = [&](int span) {
        const uint32_t own = lane_here(), shift = own >> 5 << 3;
        lds_words *ps = lds_pointer(lds_at(&lds.scale[0][0][0]) + (uint32_t)((span >> 1) & 1) * (uint32_t)sizeof(lds.scale[0]) +
                                    16u * (uint32_t)(span & 1) + (own & 31u) * 32u);
#pragma unroll
        for (int k = 0; k < kMB; ++k)
            xs[k] = ps[(wm * kMB + k) * 64];
#pragma unroll
        for (int k = 0; k < kNB; ++k)
            ws[k] = ps[(kBM + wn * kNB + k) * 64];
        // a word holds 4 chunks' scales: the lane's are bytes 0 and 2 of these
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int k = 0; k < kMB; ++k)
                xs[k][q] >>= shift;
#pragma unroll
            for (int k = 0; k < kNB; ++k)
                ws[k][q] >>= shift;
        }
    };
    // the products of quarter kQ of a span's step kS
    auto multiply = [&](auto s, auto q) {
        constexpr int kS = decltype(s)::value, kQ = decltype(q)::value, kWord = 2 * kS + kQ / 2, kByte = kQ % 2 * 2;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kNB; ++j)
#pragma unroll
            for (int k = 0; k < kMB; ++k)
                acc[k][j] = mma32<kByte>(w[kQ & 1][j], x[kQ & 1][k], acc[k][j], ws[j][kWord], xs[k][kWord]);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto landed = [&]() {
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((kRing - 2) * kPer));
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        barrier_no_fence();
    };
    auto step = [&](int span, auto s, auto tail) {
        constexpr int kS = decltype(s)::value;
        const int at = 2 * span + kS;
        hold(ax, aw, row);
        using Z = std::integral_constant<int, 0>;
        using I = std::integral_constant<int, 1>;
        using II = std::integral_constant<int, 2>;
        using III = std::integral_constant<int, 3>;
        const int buf = (at - 2 * p0) % kRing, other = (at - 2 * p0 + 1) % kRing;
        read(at, buf, 1, tail);
        multiply(s, Z());
        read(at, buf, 2, tail);
        multiply(s, I());
        read(at, buf, 3, tail);
        multiply(s, II());
        // all have read this buffer, and the next step's has landed
        landed();
        if (!kWhole && kS == 0)
            store_scales(span + 1 - p0);       // asked for a step ago; read behind the next barrier
        load(at + kRing, buf);
        if (kWhole && kS == 0 && (span - p0) % 2 == 0)
            copy_scales(span + 2, ((span - p0) / 2 + 1) & 1);
        if (!kWhole && kS == 1)
            load_scales(span + 2);
        read(at + 1, other, 0, std::integral_constant<bool, kS == 1 || decltype(tail)::value>());
        multiply(s, III());
        if (kS == 1)
            read_scales(span + 1 - p0);
    };
    // The epilogue's place: four columns of a row per lane.
    constexpr int kLanes = kCols / 4, kStep = 64 / kLanes, kIter = 32 / kStep;   // lanes of a row; rows at a time
    const int c4 = (lane % kLanes) * 4, n = n0 + wn * kCols + c4, lr = lane / kLanes;
    const int mw = m0 + wm * kMB * 32;
    // The usual case handles four columns at a time, with a 16-bit residual or
    // none; rows that end inside a lane's four columns, and binary32 residuals,
    // go element by element.
    const bool wide = !a.parts && a.N % 4 == 0 && (!a.residual || a.dtype != INT4VH_ROWS_F32);
    const bool early = wide && a.residual;
    // The usual residual is asked for up front: it takes a memory's latency.
    Pair2 res[kMB][kIter];
    if (early)
#pragma unroll
        for (int i = 0; i < kMB; ++i)
#pragma unroll
            for (int k = 0; k < kIter; ++k) {
                const int m = min(mw + i * 32 + lr + k * kStep, a.M - 1);
                res[i][k] = *reinterpret_cast<const Pair2 *>(static_cast<const uint16_t *>(a.residual) +
                                                             (size_t)m * a.residual_stride + min(n, a.N - 4));
            }
    if (kWhole) {
        copy_scales(p0, 0);
    } else {
        load_scales(p0);
        store_scales(0);
        load_scales(p0 + 1);
    }
#pragma unroll
    for (int i = 0; i < kRing; ++i)
        load(2 * p0 + i, i);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm((kRing - 1) * kPer));
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    barrier_no_fence();
    read_scales(0);
    read(2 * p0, 0, 0, std::true_type());
    // whole spans: quarters past K multiply zeros (a way out of the middle of a
    // span would copy all sums); only the last span can have any
    for (int span = p0; span < (kWhole ? p1 : p1 - 1); ++span) {
        step(span, std::integral_constant<int, 0>(), std::false_type());
        step(span, std::integral_constant<int, 1>(), std::false_type());
    }
    if (!kWhole) {
        step(p1 - 1, std::integral_constant<int, 0>(), std::true_type());
        if (16 * (p1 - 1) + 8 < blocks)
            step(p1 - 1, std::integral_constant<int, 1>(), std::true_type());
    }

    // D: column = activation row lane & 31, rows = weight rows 8 (r / 4) + 4 (lane /
    // 32) + r % 4.  Each wave turns its sums around in LDS, 32 activation rows at a
    // time, so that its lanes hold four columns of a row and rows are written whole.
    float *turn = reinterpret_cast<float *>(mem) + wave * kArea;
    // Bias and activation where the sums are: what is executed once for every four
    // outputs below stays short (with the activations there, every one of its
    // copies was an instruction cache miss, 3 us a block of sums).
    if (!a.parts) {
        if (a.bias)
#pragma unroll
            for (int j = 0; j < kNB; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float b = column_bias(a, min(n0 + (wn * kNB + j) * 32 + 8 * (r / 4) + 4 * half + r % 4, a.N - 1));
#pragma unroll
                    for (int i = 0; i < kMB; ++i)
                        acc[i][j][r] += b;
                }
        if (a.activation != INT4VH_ACT_NONE)
#pragma unroll
            for (int i = 0; i < kMB; ++i)
#pragma unroll
                for (int j = 0; j < kNB; ++j) {
                    float y[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        y[r] = acc[i][j][r];
                    activate(y, a.activation);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        acc[i][j][r] = y[r];
                }
    }
    __builtin_amdgcn_s_waitcnt(0);
    barrier_no_fence();                                        // the last step's reads and copies are done
    // sums of 32 activation rows, turned
    auto turn_rows = [&](int i) {
#pragma unroll
        for (int j = 0; j < kNB; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4 *>(turn + n32 * kPitch + j * 32 + 8 * q + 4 * half) =
                    f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        wave_fence();
    };
    auto write_wide = [&](auto dtype) {
        constexpr int kDtype = decltype(dtype)::value;
        constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;
#pragma unroll
        for (int i = 0; i < kMB; ++i) {
            turn_rows(i);
            const int m = mw + i * 32 + lr;
            char *to = static_cast<char *>(a.out) + ((size_t)m * a.out_stride + n) * kSize;
#pragma unroll
            for (int k = 0; k < kIter; ++k) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(turn + (lr + k * kStep) * kPitch + c4);
                if (m + k * kStep < a.M && n < a.N)
                    store_four<kDtype>(to, v, early, make_uint2(res[i][k].w[0], res[i][k].w[1]));
                to += (size_t)kStep * a.out_stride * kSize;
            }
            wave_fence();
        }
    };
    if (wide) {
        if (a.dtype == INT4VH_ROWS_F16)
            write_wide(std::integral_constant<int, INT4VH_ROWS_F16>());
        else if (a.dtype == INT4VH_ROWS_BF16)
            write_wide(std::integral_constant<int, INT4VH_ROWS_BF16>());
        else
            write_wide(std::integral_constant<int, INT4VH_ROWS_F32>());
        return;
    }
#pragma unroll
    for (int i = 0; i < kMB; ++i) {
        const int mi = mw + i * 32;
        turn_rows(i);
        if (a.parts) {
#pragma nounroll
            for (int r = lr; r < 32; r += kStep)
                if (mi + r < a.M && n < a.N)
                    *reinterpret_cast<f32x4 *>(&a.parts[((size_t)part * a.M + mi + r) * a.n_pad + n]) =
                        *reinterpret_cast<const f32x4 *>(turn + r * kPitch + c4);
        } else {
#pragma nounroll
            for (int e = lane; e < 32 * kCols; e += 64) {
                const int m = mi + e / kCols, c = n0 + wn * kCols + e % kCols;
                if (m < a.M && c < a.N)
                    store_one(a, m, c, turn[e / kCols * kPitch + e % kCols]);
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

// Spans of 512 channels that parts of K have to save a workgroup.
constexpr int kSplitGain = 7;

// How a call of these sizes runs.
enum Kind { kStream, kTile64, kTile128 };      // tiles of 64, 128 rows x 128 columns
struct Plan {
    Kind kind;
    int splits, split_spans;                   // parts of K, and spans of 512 channels in each
    int tiles_m, tiles_n;
};

long long tiles_of(int M, int N, int bm)
{
    return (long long)((M + bm - 1) / bm) * ((N + 127) / 128);
}

Plan plan_for(int M, int N, int K, int cus)
{
    Plan p;
    const int spans = (K + 511) / 512;
    p.splits = 1;
    if (M <= 16) {
        p.kind = kStream;
        p.tiles_m = 1;
        p.tiles_n = (N + 15) / 16;
        p.splits = (K + kSMaxK - 1) / kSMaxK;
    } else {
        p.kind = 2 * tiles_of(M, N, 128) >= cus ? kTile128 : kTile64;
        const int bm = p.kind == kTile128 ? 128 : 64;
        p.tiles_m = (M + bm - 1) / bm;
        p.tiles_n = (N + 127) / 128;
        // Few tiles: parts of K, up to a workgroup a compute unit, where that takes
        // kSplitGain spans out of a workgroup's way.  A span is about 1 us, and
        // writing and joining the parts cost about 6: 64 x 5120 x 17408 takes 29.2 us
        // whole and 16.3 in 4 parts, 17 x 5120 x 5120 12.1 and 10.5, but
        // 128 x 5120 x 5120 12.8 whole and 14.6 in 2.
        if (p.kind == kTile64) {
            int s = 1;
            while (2 * s * tiles_of(M, N, 64) <= cus && spans / (2 * s) >= 2)
                s *= 2;
            if (spans - (spans + s - 1) / s >= kSplitGain)
                p.splits = s;
        }
    }
    p.split_spans = (spans + p.splits - 1) / p.splits;
    p.splits = (spans + p.split_spans - 1) / p.split_spans;
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

template <bool kWhole>
void launch_stream(const MxArgs &a, dim3 grid, hipStream_t s)
{
    const int per_wave = (4 * a.split_spans + kSWaves - 1) / kSWaves;
    const dim3 block(kSThreads);
    if (per_wave <= 1)
        hipLaunchKernelGGL((mx_stream_kernel<1, kWhole>), grid, block, 0, s, a);
    else if (per_wave <= 2)
        hipLaunchKernelGGL((mx_stream_kernel<2, kWhole>), grid, block, 0, s, a);
    else if (per_wave <= 3)
        hipLaunchKernelGGL((mx_stream_kernel<3, kWhole>), grid, block, 0, s, a);
    else if (per_wave <= 4)
        hipLaunchKernelGGL((mx_stream_kernel<4, kWhole>), grid, block, 0, s, a);
    else if (per_wave <= 5)
        hipLaunchKernelGGL((mx_stream_kernel<5, kWhole>), grid, block, 0, s, a);
    else if (per_wave <= 6)
        hipLaunchKernelGGL((mx_stream_kernel<6, kWhole>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((mx_stream_kernel<8, kWhole>), grid, block, 0, s, a);
}

template <int kWM, int kWN, int kMB, int kNB, int kRing>
void launch_tiles(const MxArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((long long)a.tiles_m * a.tiles_n * a.splits)), block(64 * kWM * kWN);
    if (a.K % 512 == 0 && rows_aligned(a.x_scales, 16) && rows_aligned(a.w_scales, 16))
        hipLaunchKernelGGL((mx_tile_kernel<kWM, kWN, kMB, kNB, kRing, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((mx_tile_kernel<kWM, kWN, kMB, kNB, kRing, false>), grid, block, 0, s, a);
}

constexpr long long kGridThreads = 1ll << 31;

template <int kDtype>
void launch_quantize(const void *x, int64_t x_stride, int M, int H, uint8_t *codes, uint8_t *scales, hipStream_t s)
{
    // one long row, unless it would take more threads than a grid may have
    const bool flat = M == 1 || (x_stride == H && (long long)M * H / 8 <= kGridThreads);
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
    const long long threads = chunks < kGridThreads ? chunks : kGridThreads;
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<kDtype>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s,
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
    a.split_spans = p.split_spans;
    a.tiles_m = p.tiles_m;
    a.tiles_n = p.tiles_n;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 stream_grid(p.tiles_n < 2 * cus ? p.tiles_n : 2 * cus, p.splits);
    if (p.kind == kStream && K % 128 == 0)
        launch_stream<true>(a, stream_grid, s);
    else if (p.kind == kStream)
        launch_stream<false>(a, stream_grid, s);
    else if (p.kind == kTile64)
        launch_tiles<2, 2, 1, 2, 3>(a, s);
    else
        launch_tiles<2, 2, 2, 2, 2>(a, s);
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
