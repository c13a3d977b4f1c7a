// logits.hip -- rules on logits (penalties for repeated tokens, biases,
// grammar masks) and verification under them, for MI355X (gfx950); formulas
// and order of rounding in int4vh_logits.h.
//
// Bound by HBM: the logits are read once (and written once by the apply
// call); a row of 151936 binary32 logits is 608 KB against a few KB of rules.
// The rules' cost is finding each token's count, which depends on the request
// and hardly on the row: a workgroup takes a slice of the vocabulary and
// several rows of ONE request, counts the slice's tokens of the request's
// history in LDS (integer atomics: any order gives the same counts), and then
// walks its rows; a row's draft is counted for the rows behind it.  The
// history is read once per slice and row group, from L2.
//
// Verification keeps one pass over the logits: each wave reduces 1024 tokens
// of a row, held in registers (16 per lane), to the best keys, (max, sum) and
// the draft's logit; rules_merge_kernel joins the chunks of each row and
// counts accepted drafts.  A chunk's top-k goes by a threshold: the k-th
// largest of the 64 lanes' maxima is at most the chunk's k-th value, so the
// few values that reach it are the candidates; they are ranked by counting
// the larger ones.  Everything is exact, ties included (keys are distinct).
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>

#include "int4vh.h"
#include "int4vh_internal.h"
#include "int4vh_logits.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace {

using namespace int4vh_detail;

typedef unsigned long long u64;

constexpr int kChunk = 1024;              // tokens of a row per wave
constexpr int kPer = kChunk / 64;         // tokens per lane: 4 at a time, 256 apart
constexpr int kMaxWaves = 8;
constexpr int kMaxTopK = 16;
constexpr int kMaxRows = 4096;
constexpr int kBuf = 128;                 // candidate keys per wave
constexpr float kNegInf = -__builtin_huge_valf();
constexpr uint32_t kSeen = 0x80000000u;   // count word: in the history's prompt; low bits: times generated

struct RulesArgs {
    const void *logits;
    long long logits_stride;
    const int32_t *draft;      // [R, T-1] or null
    int R, T, V;
    int4vh_logit_rules r;      // zeros for none
    int has_penalty, has_bias;
    int row_group;             // rows per workgroup
    // apply
    void *out;
    long long out_stride;
    // verify
    int top_k, n_chunks;
    float lse_scale;           // log2(e) / temperature
    u64 *heads;                // [R*T, n_chunks] best key of each chunk, 0 if none
    u64 *lists;                // [R*T, n_chunks, top_k] best keys, best first, 0 past the last
    float2 *sums;              // [R*T, n_chunks] (max, sum of exp2((x - max) * lse_scale))
    float *draft_logit;        // [R*T] ruled logit of the row's draft, where it is in [0, V)
};

// Key of a (value, token) pair whose unsigned order is: larger value, then
// lower token.  -0 is keyed as +0; key 0 is below every pair's.
__device__ __forceinline__ uint32_t order_word(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ u64 order_key(float v, int token)
{
    return ((u64)order_word(v) << 32) | (u64)(~(uint32_t)token);
}
__device__ __forceinline__ float key_value(u64 k)
{
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ int key_token(u64 k)
{
    return (int)(~(uint32_t)k);
}

__device__ __forceinline__ u64 shfl_xor64(u64 k, int mask)
{
    const uint32_t lo = __shfl_xor((uint32_t)k, mask), hi = __shfl_xor((uint32_t)(k >> 32), mask);
    return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ u64 wave_max64(u64 k)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const u64 o = shfl_xor64(k, off);
        k = o > k ? o : k;
    }
    return k;
}
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v = fmaxf(v, __shfl_xor(v, off));
    return v;
}
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
}

// exp2((x - m) * scale) of a value at most m; 1 at the maximum itself, so that
// infinities do not meet, and 0 for -infinity and NaN.
__device__ __forceinline__ float exp2_below(float x, float m, float scale)
{
    return x == m ? 1.0f : x > kNegInf ? exp2f((x - m) * scale) : 0.0f;
}

// LDS written and read by one wave alone: its accesses execute in order, so
// only the compiler has to be held back.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// Keeps the k best of the n (<= kBuf) distinct keys buf[0, n), best first, and
// returns how many there are (min(n, k)).  A key's rank is the number of
// larger ones.  Called by a whole wave on its own buffer.
__device__ __forceinline__ int keep_best(volatile u64 *buf, int n, int k, int lane)
{
    const u64 a = lane < n ? buf[lane] : 0ull, b = lane + 64 < n ? buf[lane + 64] : 0ull;
    int ra = 0, rb = 0;
    for (int i = 0; i < n; ++i) {
        const u64 o = buf[i];
        ra += o > a;
        rb += o > b;
    }
    wave_fence();
    if (lane < n && ra < k)
        buf[ra] = a;
    if (lane + 64 < n && rb < k)
        buf[rb] = b;
    wave_fence();
    return n < k ? n : k;
}

// Appends the keys of the lanes in `mask`; a buffer that could overflow is
// first cut to its k best.  Wave-uniform control flow.
__device__ __forceinline__ void push(volatile u64 *buf, int &n, u64 key, u64 mask, int k, int lane)
{
    if (n + __popcll(mask) > kBuf) {
        n = keep_best(buf, n, k, lane);
        if (n == k) {
            const u64 last = buf[k - 1];
            mask &= __ballot(key > last);
        }
    }
    if (mask >> lane & 1ull)
        buf[n + __popcll(mask & ((1ull << lane) - 1ull))] = key;
    wave_fence();
    n += __popcll(mask);
}

// A word th (at least 1) that at least k lanes' words reach, and where it can
// be no more than k + 8; 1 where fewer than k lanes have a word, since then
// lower values of the same lanes are wanted too.  Bits are set from the top
// while enough lanes still reach the word.
__device__ __forceinline__ uint32_t reach_threshold(uint32_t word, int k)
{
    uint32_t th = 0u;
    if (__popcll(__ballot(word != 0u)) < k)
        return 1u;
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
        const int c = __popcll(__ballot(word >= (th | bit)));
        if (c >= k) {
            th |= bit;
            if (c <= k + 8)
                break;
        }
    }
    return th ? th : 1u;
}

// Four consecutive logits token .. token+3 of a row (-infinity past V).
template <int kDtype>
__device__ __forceinline__ void load4(const void *row, int token, int V, float (&v)[4])
{
    if (token + 4 <= V) {
        if constexpr (kDtype == INT4VH_ROWS_F32) {
            const Words4 w = *reinterpret_cast<const Words4 *>(static_cast<const float *>(row) + token);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = __uint_as_float(w.w[j]);
        } else {
            const Pair2 w = *reinterpret_cast<const Pair2 *>(static_cast<const uint16_t *>(row) + token);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = from_bits16((w.w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, kDtype);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = kNegInf;
            if (token + j < V) {
                if constexpr (kDtype == INT4VH_ROWS_F32)
                    v[j] = static_cast<const float *>(row)[token + j];
                else
                    v[j] = from_bits16(static_cast<const uint16_t *>(row)[token + j], kDtype);
            }
        }
    }
}

template <int kDtype>
__device__ __forceinline__ void store4(void *row, int token, int V, const float (&v)[4])
{
    if constexpr (kDtype == INT4VH_ROWS_F32) {
        float *p = static_cast<float *>(row) + token;
        if (token + 4 <= V) {
            Words4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w.w[j] = __float_as_uint(v[j]);
            *reinterpret_cast<Words4 *>(p) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (token + j < V)
                    p[j] = v[j];
        }
    } else {
        uint16_t *p = static_cast<uint16_t *>(row) + token;
        if (token + 4 <= V) {
            Pair2 w;
            w.w[0] = to_bits16(v[0], kDtype) | (to_bits16(v[1], kDtype) << 16);
            w.w[1] = to_bits16(v[2], kDtype) | (to_bits16(v[3], kDtype) << 16);
            *reinterpret_cast<Pair2 *>(p) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (token + j < V)
                    p[j] = (uint16_t)to_bits16(v[j], kDtype);
        }
    }
}

__device__ __forceinline__ long long clamp64(long long v, long long lo, long long hi)
{
    return v < lo ? lo : v > hi ? hi : v;
}

// The slice's counts and biases of one request, with the drafts in front of
// row t0 counted.  cnt: words (kSeen | times generated) of tokens base ..
// base + S - 1; bias: their biases.  Called by the whole workgroup, which
// waits at the end.
__device__ __forceinline__ void prepare_slice(const RulesArgs &a, int req, int t0, int base, int S, uint32_t *cnt,
                                              float *bias)
{
    const int tid = threadIdx.x, nt = blockDim.x;
    if (a.has_penalty)
        for (int i = tid; i < S; i += nt)
            cnt[i] = 0u;
    uint32_t *order = reinterpret_cast<uint32_t *>(bias);
    if (a.has_bias)
        for (int i = tid; i < S; i += nt)
            order[i] = 0u;
    __syncthreads();
    if (a.has_penalty) {
        if (a.r.history) {
            const long long b = clamp64(a.r.history_offsets[req], 0, a.r.n_history);
            const long long e = clamp64(a.r.history_offsets[req + 1], 0, a.r.n_history);
            const long long made = b + (a.r.n_prompt ? a.r.n_prompt[req] : 0);
            constexpr int kFly = 8;                 // loads in flight per thread
            for (long long i0 = b + tid; i0 < e; i0 += (long long)nt * kFly) {
                int32_t v[kFly];
#pragma unroll
                for (int u = 0; u < kFly; ++u) {
                    const long long i = i0 + (long long)u * nt;
                    v[u] = i < e ? a.r.history[i] : -1;
                }
#pragma unroll
                for (int u = 0; u < kFly; ++u) {
                    const uint32_t at = (uint32_t)v[u] - (uint32_t)base;
                    if (v[u] >= 0 && at < (uint32_t)S) {
                        if (i0 + (long long)u * nt < made)
                            atomicOr(&cnt[at], kSeen);
                        else
                            atomicAdd(&cnt[at], 1u);
                    }
                }
            }
        }
        if (tid < t0) {
            const int d = a.draft[(size_t)req * (a.T - 1) + tid];
            const uint32_t at = (uint32_t)d - (uint32_t)base;
            if (d >= 0 && at < (uint32_t)S)
                atomicAdd(&cnt[at], 1u);
        }
    }
    if (a.has_bias) {
        // the last entry of an id holds: the largest entry number, then, each
        // thread at its own tokens, that entry's value
        const long long b = clamp64(a.r.bias_offsets[req], 0, a.r.n_bias);
        const long long e = clamp64(a.r.bias_offsets[req + 1], 0, a.r.n_bias);
        for (long long i = b + tid; i < e; i += nt) {
            const int32_t v = a.r.bias_ids[i];
            const uint32_t at = (uint32_t)v - (uint32_t)base;
            if (v >= 0 && at < (uint32_t)S)
                atomicMax(&order[at], (uint32_t)(i - b) + 1u);
        }
        __syncthreads();
        for (int i = tid; i < S; i += nt) {
            const uint32_t o = order[i];
            bias[i] = o ? a.r.bias_values[b + (o - 1u)] : 0.0f;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float penalise(float l, uint32_t word, float rep, float freq, float pres)
{
    const uint32_t count = word & ~kSeen;
    float x = l > 0.0f ? l / rep : l * rep;
    x = x - freq * (float)count;
    return x - (count ? pres : 0.0f);
}

// Grid (slices of the vocabulary, requests, row groups); each wave takes a
// chunk of kChunk tokens.  kVerify: reduce the rows; otherwise write them out.
template <int kDtype, bool kVerify, bool kTopK, bool kLse>
__global__ void __launch_bounds__(64 * kMaxWaves) rules_kernel(RulesArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint32_t s_mem[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n_waves = blockDim.x >> 6;
    const int S = n_waves * kChunk;
    uint32_t *cnt = s_mem;
    float *bias = reinterpret_cast<float *>(s_mem + (a.has_penalty ? S : 0));
    volatile u64 *buf = reinterpret_cast<u64 *>(s_mem + (a.has_penalty ? S : 0) + (a.has_bias ? S : 0)) + wave * kBuf;
    const int base = blockIdx.x * S;
    const int req = blockIdx.y;
    const int t0 = blockIdx.z * a.row_group, t1 = min(a.T, t0 + a.row_group);
    const int V = a.V;

    if (a.has_penalty || a.has_bias)
        prepare_slice(a, req, t0, base, S, cnt, bias);
    const int chunk0 = base + wave * kChunk;
    if (chunk0 >= V)
        return;                               // no barrier follows
    const int chunk = chunk0 / kChunk;
    uint32_t *my_cnt = cnt + wave * kChunk;
    const float *my_bias = bias + wave * kChunk;
    const float rep = a.r.repetition ? a.r.repetition[req] : 1.0f;
    const float freq = a.r.frequency ? a.r.frequency[req] : 0.0f;
    const float pres = a.r.presence ? a.r.presence[req] : 0.0f;
    constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;

    for (int t = t0; t < t1; ++t) {
        const int row = req * a.T + t;
        const char *lrow = static_cast<const char *>(a.logits) + (size_t)row * a.logits_stride * kSize;
        const uint32_t *mask = nullptr;
        bool none = false;                    // nothing is allowed
        if (a.r.mask) {
            const long long mi = a.r.mask_index ? a.r.mask_index[row] : row;
            none = mi >= a.r.n_masks;
            if (mi >= 0 && !none)
                mask = a.r.mask + (size_t)mi * a.r.mask_stride;
        }
        const int d = t < a.T - 1 ? a.draft[(size_t)req * (a.T - 1) + t] : -1;

        float x[kPer / 4][4];
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i)
            load4<kDtype>(lrow, chunk0 + 256 * i + 4 * lane, V, x[i]);
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) {
            const int at = 256 * i + 4 * lane, token = chunk0 + at;
            if (a.has_penalty) {
                const uint4 c = *reinterpret_cast<const uint4 *>(my_cnt + at);
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                if ((c.x | c.y | c.z | c.w) != 0u) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (w[j])
                            x[i][j] = penalise(x[i][j], w[j], rep, freq, pres);
                }
            }
            if (a.has_bias) {
                const float4 b = *reinterpret_cast<const float4 *>(my_bias + at);
                x[i][0] += b.x;
                x[i][1] += b.y;
                x[i][2] += b.z;
                x[i][3] += b.w;
            }
            if (mask || none) {
                const uint32_t bits = mask && token < V ? mask[token >> 5] >> (token & 31) : 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i][j] = (bits >> j) & 1u ? x[i][j] : kNegInf;
            }
        }
        if constexpr (!kVerify) {
            char *orow = static_cast<char *>(a.out) + (size_t)row * a.out_stride * kSize;
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i)
                store4<kDtype>(orow, chunk0 + 256 * i + 4 * lane, V, x[i]);
        } else {
            // tokens past V are -infinity here: biases do not reach them
            float best = kNegInf;             // fmaxf passes over NaN
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    best = fmaxf(best, x[i][j]);
            const size_t slot = (size_t)row * a.n_chunks + chunk;
            if constexpr (kLse) {
                const float m = wave_max(best);
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < kPer / 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s += exp2_below(x[i][j], m, a.lse_scale);
                s = wave_sum(s);
                if (lane == 0)
                    a.sums[slot] = make_float2(m, m > kNegInf ? s : 0.0f);
            }
            if constexpr (kTopK) {
                const int k = a.top_k;
                const uint32_t th = reach_threshold(best > kNegInf ? order_word(best) : 0u, k);
                int n = 0;
#pragma unroll
                for (int i = 0; i < kPer / 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool take = x[i][j] > kNegInf && order_word(x[i][j]) >= th;
                        const u64 m = __ballot(take);
                        if (m)
                            push(buf, n, order_key(x[i][j], chunk0 + 256 * i + 4 * lane + j), m, k, lane);
                    }
                n = keep_best(buf, n, k, lane);
                const u64 key = lane < n ? buf[lane] : 0ull;
                if (lane < k)
                    a.lists[slot * k + lane] = key;
                if (lane == 0)
                    a.heads[slot] = key;
            } else {
                u64 key = 0ull;
#pragma unroll
                for (int i = 0; i < kPer / 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u64 o = x[i][j] > kNegInf ? order_key(x[i][j], chunk0 + 256 * i + 4 * lane + j) : 0ull;
                        key = o > key ? o : key;
                    }
                key = wave_max64(key);
                if (lane == 0)
                    a.heads[slot] = key;
            }
            const uint32_t da = (uint32_t)d - (uint32_t)chunk0;
            if (d >= 0 && d < V && da < (uint32_t)kChunk && (int)((da >> 2) & 63u) == lane) {
                float v = kNegInf;
#pragma unroll
                for (int i = 0; i < kPer / 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v = (int)(da >> 8) == i && (int)(da & 3u) == j ? x[i][j] : v;
                a.draft_logit[row] = v;
            }
        }
        // the rows behind this one count its draft: this wave's own words
        if (a.has_penalty && t + 1 < t1) {
            const uint32_t da = (uint32_t)d - (uint32_t)chunk0;
            if (d >= 0 && da < (uint32_t)kChunk && lane == 0)
                my_cnt[da] += 1u;
            wave_fence();
        }
    }
}

struct MergeArgs {
    const u64 *heads, *lists;
    const float2 *sums;
    const float *draft_logit;
    const int32_t *draft;
    const float *draft_probs, *uniforms;   // both or neither
    int R, T, V, top_k, n_chunks;
    float temperature, lse_scale;
    float *logits_max;
    int32_t *argmax, *topk_ids;
    float *topk_logits, *lse, *p_draft;
    int32_t *n_acc;
};

// One workgroup per request, one wave per row: the row's chunks joined, then
// the request's accepted count.
template <bool kTopK, bool kLse>
__global__ void __launch_bounds__(64 * 16) rules_merge_kernel(MergeArgs a)
{
    __shared__ u64 s_buf[16][kBuf];
    __shared__ int s_ok[16];
    const int lane = threadIdx.x & 63, t = threadIdx.x >> 6, req = blockIdx.x;
    const int row = req * a.T + t;
    const int n_chunks = a.n_chunks;
    const u64 *heads = a.heads + (size_t)row * n_chunks;
    const bool drafted = t < a.T - 1;
    const size_t di = drafted ? (size_t)req * (a.T - 1) + t : 0;
    const int d = drafted ? a.draft[di] : -1;

    float gm = kNegInf, gs = 0.0f;
    if constexpr (kLse) {
        const float2 *sums = a.sums + (size_t)row * n_chunks;
        for (int c = lane; c < n_chunks; c += 64)
            gm = fmaxf(gm, sums[c].x);
        gm = wave_max(gm);
        for (int c = lane; c < n_chunks; c += 64) {
            const float2 p = sums[c];
            gs += p.y * exp2_below(p.x, gm, a.lse_scale);
        }
        gs = wave_sum(gs);
        if (a.lse && lane == 0)
            a.lse[row] = gs > 0.0f ? gm / a.temperature + logf(gs) : kNegInf;
    }

    u64 best = 0ull;                          // of this lane's chunks
    for (int c = lane; c < n_chunks; c += 64) {
        const u64 h = heads[c];
        best = h > best ? h : best;
    }
    float p = 0.0f;
    u64 top;                                  // the row's best key
    if constexpr (kTopK) {
        volatile u64 *buf = s_buf[t];
        const int k = a.top_k;
        const uint32_t th = reach_threshold((uint32_t)(best >> 32), k);
        int n = 0;
        for (int c0 = 0; c0 < n_chunks; c0 += 64) {
            const int c = c0 + lane;
            const u64 h = c < n_chunks ? heads[c] : 0ull;
            // the lists whose best key reaches the threshold, a lane each
            const bool open = h != 0ull && (uint32_t)(h >> 32) >= th;
            if (!__ballot(open))
                continue;
            const u64 *list = a.lists + ((size_t)row * n_chunks + (open ? c : 0)) * k;
            for (int j = 0; j < k; ++j) {
                const u64 key = open ? list[j] : 0ull;
                const u64 m = __ballot(key != 0ull && (uint32_t)(key >> 32) >= th);
                if (!m)
                    break;                    // lists are best first
                push(buf, n, key, m, k, lane);
            }
        }
        n = keep_best(buf, n, k, lane);
        const u64 key = lane < n ? buf[lane] : 0ull;
        top = n ? buf[0] : 0ull;
        const float v = key ? key_value(key) : kNegInf;
        const int id = key ? key_token(key) : -1;
        if (lane < k) {
            a.topk_ids[(size_t)row * k + lane] = id;
            a.topk_logits[(size_t)row * k + lane] = v;
        }
        if (a.draft_probs && drafted) {
            const float m = key_value(top);
            const float e = key ? exp2_below(v, m, a.lse_scale) : 0.0f;
            const float sum = wave_sum(e), e_d = wave_sum(key && id == d ? e : 0.0f);
            p = n ? e_d / sum : 0.0f;
        }
    } else {
        top = wave_max64(best);
        if (kLse && a.draft_probs && drafted && d >= 0 && d < a.V && gs > 0.0f)
            p = exp2_below(a.draft_logit[row], gm, a.lse_scale) / gs;
    }
    const int id = top ? key_token(top) : -1;
    if (lane == 0) {
        a.argmax[row] = id;
        a.logits_max[row] = top ? key_value(top) : kNegInf;
        bool ok = false;
        if (drafted) {
            if (a.draft_probs) {
                a.p_draft[di] = p;
                ok = a.uniforms[di] * a.draft_probs[di] < p;
            } else {
                ok = id >= 0 && id == d;
            }
        }
        s_ok[t] = ok;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        while (n < a.T - 1 && s_ok[n])
            ++n;
        a.n_acc[req] = n;
    }
}

// ---------------------------------------------------------------- host side

struct Layout {
    size_t heads, lists, sums, draft_logit, bytes;
    int n_chunks;
};

size_t round256(size_t n)
{
    return (n + 255) / 256 * 256;
}

Layout layout_for(int R, int T, int V, int top_k)
{
    Layout l;
    const size_t M = (size_t)R * T;
    l.n_chunks = (V + kChunk - 1) / kChunk;
    l.heads = 0;
    l.lists = round256(M * l.n_chunks * 8);
    l.sums = l.lists + round256(M * l.n_chunks * 8 * top_k);
    l.draft_logit = l.sums + round256(M * l.n_chunks * 8);
    l.bytes = l.draft_logit + round256(M * 4);
    return l;
}

bool sizes_ok(int R, int T, int V)
{
    return R >= 1 && T >= 1 && T <= INT4VH_MAX_T && V >= 1 && (long long)R * T <= kMaxRows;
}

constexpr int kMaxV = 1 << 24;

int check(const void *logits, int64_t stride, int dtype, const int32_t *draft, int R, int T, int V,
          const int4vh_logit_rules *r)
{
    if (!sizes_ok(R, T, V) || !rows_known(dtype) || !logits || (T > 1 && !draft))
        return INT4VH_EINVAL;
    if (R * T > 1 && stride < V)
        return INT4VH_EINVAL;
    if (r) {
        if (r->n_history < 0 || r->n_bias < 0 || (r->n_history > 0 && !r->history) || (r->history && !r->history_offsets))
            return INT4VH_EINVAL;
        if (r->bias_ids && (!r->bias_values || !r->bias_offsets))
            return INT4VH_EINVAL;
        if (r->n_bias > 0 && !r->bias_ids)
            return INT4VH_EINVAL;
        if (r->mask && (r->n_masks < 1 || r->mask_stride < (V + 31) / 32 || (!r->mask_index && r->n_masks < R * T)))
            return INT4VH_EINVAL;
        if (!r->mask && r->mask_index)
            return INT4VH_EINVAL;
    }
    if (!rows_aligned(logits, rows_size(dtype)) || !rows_aligned(draft, 4))
        return INT4VH_EALIGN;
    if (r && (!rows_aligned(r->history, 4) || !rows_aligned(r->history_offsets, 8) || !rows_aligned(r->n_prompt, 4) ||
              !rows_aligned(r->repetition, 4) || !rows_aligned(r->frequency, 4) || !rows_aligned(r->presence, 4) ||
              !rows_aligned(r->bias_ids, 4) || !rows_aligned(r->bias_values, 4) || !rows_aligned(r->bias_offsets, 8) ||
              !rows_aligned(r->mask, 4) || !rows_aligned(r->mask_index, 4)))
        return INT4VH_EALIGN;
    return V > kMaxV ? INT4VH_EUNSUPPORTED : INT4VH_OK;
}

void fill_rules(RulesArgs &a, const int4vh_logit_rules *r, int T)
{
    a.r = r ? *r : int4vh_logit_rules{};
    const bool any = a.r.repetition || a.r.frequency || a.r.presence;
    a.has_penalty = any && (a.r.history || T > 1);
    a.has_bias = a.r.bias_ids != nullptr;
}

struct Shape {
    dim3 grid, block;
    size_t lds;
};

Shape shape_for(RulesArgs &a, bool topk, int cus)
{
    const int n_chunks = (a.V + kChunk - 1) / kChunk;
    const int waves = n_chunks < kMaxWaves ? n_chunks : kMaxWaves;
    const int slices = (n_chunks + waves - 1) / waves;
    // rows of one workgroup share its counts; few requests: fewer rows each,
    // so that two workgroups a compute unit are there
    int groups = 1;
    while (groups < a.T && (long long)slices * a.R * groups < 2ll * cus)
        ++groups;
    a.row_group = (a.T + groups - 1) / groups;
    Shape s;
    s.grid = dim3(slices, a.R, (a.T + a.row_group - 1) / a.row_group);
    s.block = dim3(64 * waves);
    s.lds = (size_t)waves * kChunk * 4 * ((a.has_penalty ? 1 : 0) + (a.has_bias ? 1 : 0)) +
            (topk ? (size_t)waves * kBuf * 8 : 0);
    return s;
}

template <bool kVerify, bool kTopK, bool kLse>
hipError_t launch_rules(const RulesArgs &a, int dtype, const Shape &sh, hipStream_t s)
{
    void (*k)(RulesArgs) = dtype == INT4VH_ROWS_F32   ? rules_kernel<INT4VH_ROWS_F32, kVerify, kTopK, kLse>
                           : dtype == INT4VH_ROWS_F16 ? rules_kernel<INT4VH_ROWS_F16, kVerify, kTopK, kLse>
                                                      : rules_kernel<INT4VH_ROWS_BF16, kVerify, kTopK, kLse>;
    hipLaunchKernelGGL(k, sh.grid, sh.block, sh.lds, s, a);
    return hipGetLastError();
}

int current_cus(int *cus)
{
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e, "hipGetDevice");
    *cus = cu_count(dev);
    return INT4VH_OK;
}

int check_verify(const float *draft_probs, const float *uniforms, int T, int V, int top_k, float temperature,
                 const float *logits_max, const int32_t *argmax, const int32_t *topk_ids, const float *topk_logits,
                 const float *lse, const float *p_draft, const int32_t *n_acc)
{
    if (top_k < 0 || top_k > kMaxTopK || top_k > V || !(temperature > 0.0f) || !std::isfinite(temperature))
        return INT4VH_EINVAL;
    if (!logits_max || !argmax || !n_acc || (top_k && (!topk_ids || !topk_logits)))
        return INT4VH_EINVAL;
    if (T > 1 && ((draft_probs == nullptr) != (uniforms == nullptr) || (draft_probs && !p_draft)))
        return INT4VH_EINVAL;
    if (!rows_aligned(draft_probs, 4) || !rows_aligned(uniforms, 4) || !rows_aligned(logits_max, 4) ||
        !rows_aligned(argmax, 4) || !rows_aligned(topk_ids, 4) || !rows_aligned(topk_logits, 4) ||
        !rows_aligned(lse, 4) || !rows_aligned(p_draft, 4) || !rows_aligned(n_acc, 4))
        return INT4VH_EALIGN;
    return INT4VH_OK;
}

} // namespace

extern "C" {

int logit_rules_apply(const void *logits, int64_t logits_stride, int dtype, const int32_t *draft_ids, int R, int T,
                      int V, const int4vh_logit_rules *rules, void *out, int64_t out_stride, void *stream)
{
    if (!out || (sizes_ok(R, T, V) && R * T > 1 && out_stride < V))
        return INT4VH_EINVAL;
    int st = check(logits, logits_stride, dtype, draft_ids, R, T, V, rules);
    if (st != INT4VH_OK)
        return st;
    if (!rows_aligned(out, rows_size(dtype)))
        return INT4VH_EALIGN;
    int cus = 0;
    if ((st = current_cus(&cus)) != INT4VH_OK)
        return st;
    RulesArgs a = {};
    a.logits = logits;
    a.logits_stride = logits_stride;
    a.draft = draft_ids;
    a.R = R;
    a.T = T;
    a.V = V;
    a.out = out;
    a.out_stride = out_stride;
    fill_rules(a, rules, T);
    const Shape sh = shape_for(a, false, cus);
    const hipError_t e = launch_rules<false, false, false>(a, dtype, sh, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? INT4VH_OK : hip_fail(e, "rules kernel launch");
}

size_t logit_rules_verify_workspace_bytes(int R, int T, int V, int top_k)
{
    if (!sizes_ok(R, T, V) || V > kMaxV || top_k < 0 || top_k > kMaxTopK || top_k > V)
        return 0;
    return layout_for(R, T, V, top_k).bytes;
}

int logit_rules_verify(const void *logits, int64_t logits_stride, int dtype, const int32_t *draft_ids,
                       const float *draft_probs, const float *uniforms, int R, int T, int V,
                       const int4vh_logit_rules *rules, int top_k, float temperature, float *logits_max,
                       int32_t *argmax_ids, int32_t *topk_ids, float *topk_logits, float *lse, float *p_draft,
                       int32_t *n_accepted, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = check(logits, logits_stride, dtype, draft_ids, R, T, V, rules);
    if (st == INT4VH_EINVAL)
        return st;
    const int sv = check_verify(draft_probs, uniforms, T, V, top_k, temperature, logits_max, argmax_ids, topk_ids,
                                topk_logits, lse, p_draft, n_accepted);
    if (sv == INT4VH_EINVAL || !workspace)
        return INT4VH_EINVAL;
    if (st != INT4VH_OK)
        return st;
    if (sv != INT4VH_OK)
        return sv;
    if (!rows_aligned(workspace, 256))
        return INT4VH_EALIGN;
    const Layout l = layout_for(R, T, V, top_k);
    if (workspace_bytes < l.bytes)
        return INT4VH_EWORKSPACE;
    int cus = 0;
    if ((st = current_cus(&cus)) != INT4VH_OK)
        return st;

    char *ws = static_cast<char *>(workspace);
    const bool sampled = T > 1 && draft_probs;
    const bool want_lse = lse || (sampled && top_k == 0);
    RulesArgs a = {};
    a.logits = logits;
    a.logits_stride = logits_stride;
    a.draft = draft_ids;
    a.R = R;
    a.T = T;
    a.V = V;
    fill_rules(a, rules, T);
    a.top_k = top_k;
    a.n_chunks = l.n_chunks;
    a.lse_scale = 1.4426950408889634f / temperature;
    a.heads = reinterpret_cast<u64 *>(ws + l.heads);
    a.lists = reinterpret_cast<u64 *>(ws + l.lists);
    a.sums = reinterpret_cast<float2 *>(ws + l.sums);
    a.draft_logit = reinterpret_cast<float *>(ws + l.draft_logit);
    const Shape sh = shape_for(a, top_k > 0, cus);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (top_k)
        e = want_lse ? launch_rules<true, true, true>(a, dtype, sh, s) : launch_rules<true, true, false>(a, dtype, sh, s);
    else
        e = want_lse ? launch_rules<true, false, true>(a, dtype, sh, s)
                     : launch_rules<true, false, false>(a, dtype, sh, s);
    if (e != hipSuccess)
        return hip_fail(e, "rules kernel launch");

    MergeArgs m;
    m.heads = a.heads;
    m.lists = a.lists;
    m.sums = a.sums;
    m.draft_logit = a.draft_logit;
    m.draft = draft_ids;
    m.draft_probs = sampled ? draft_probs : nullptr;
    m.uniforms = sampled ? uniforms : nullptr;
    m.R = R;
    m.T = T;
    m.V = V;
    m.top_k = top_k;
    m.n_chunks = l.n_chunks;
    m.temperature = temperature;
    m.lse_scale = a.lse_scale;
    m.logits_max = logits_max;
    m.argmax = argmax_ids;
    m.topk_ids = topk_ids;
    m.topk_logits = topk_logits;
    m.lse = lse;
    m.p_draft = p_draft;
    m.n_acc = n_accepted;
    void (*k)(MergeArgs) = top_k ? (want_lse ? rules_merge_kernel<true, true> : rules_merge_kernel<true, false>)
                                 : (want_lse ? rules_merge_kernel<false, true> : rules_merge_kernel<false, false>);
    hipLaunchKernelGGL(k, dim3(R), dim3(64 * T), 0, s, m);
    e = hipGetLastError();
    return e == hipSuccess ? INT4VH_OK : hip_fail(e, "rules merge kernel launch");
}

size_t verify_lm_head_int4_ruled_workspace_bytes(int R, int T, int V, int H, int top_k)
{
    const size_t head = verify_lm_head_int4_workspace_bytes(R, T, V, H);
    const size_t rest = logit_rules_verify_workspace_bytes(R, T, V, top_k);
    if (!head || !rest)
        return 0;
    return round256(head) + round256((size_t)R * T * V * 4) + rest;
}

int verify_lm_head_int4_ruled(const void *hidden, const uint8_t *packed_w, const void *scales,
                              const int32_t *draft_ids, const float *draft_probs, const float *uniforms, int R, int T,
                              int V, int H, const int4vh_logit_rules *rules, int top_k, float temperature,
                              float *logits_max, int32_t *argmax_ids, int32_t *topk_ids, float *topk_logits,
                              float *lse, float *p_draft, int32_t *n_accepted, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    if (!workspace)
        return INT4VH_EINVAL;
    if (!sizes_ok(R, T, V) || H < 32 || H % 32)
        return INT4VH_EINVAL;
    // what the second half would refuse is refused before the first is launched
    char *ws = static_cast<char *>(workspace);
    int st = check(ws, V, INT4VH_ROWS_F32, draft_ids, R, T, V, rules);
    if (st == INT4VH_EINVAL)
        return st;
    const int sv = check_verify(draft_probs, uniforms, T, V, top_k, temperature, logits_max, argmax_ids, topk_ids,
                                topk_logits, lse, p_draft, n_accepted);
    if (sv == INT4VH_EINVAL || !hidden || !packed_w || !scales)
        return INT4VH_EINVAL;
    if (!rows_aligned(workspace, 256))
        return INT4VH_EALIGN;
    if (st != INT4VH_OK)
        return st;
    if (sv != INT4VH_OK)
        return sv;
    if (workspace_bytes < verify_lm_head_int4_ruled_workspace_bytes(R, T, V, H, top_k))
        return INT4VH_EWORKSPACE;
    const size_t at = round256(verify_lm_head_int4_workspace_bytes(R, T, V, H));
    float *logits = reinterpret_cast<float *>(ws + at);
    char *rest = ws + at + round256((size_t)R * T * V * 4);
    st = verify_lm_head_int4_batch(hidden, packed_w, scales, draft_ids, R, T, V, H, logits_max, argmax_ids, n_accepted,
                                   logits, workspace, at, stream);
    if (st != INT4VH_OK)
        return st;
    return logit_rules_verify(logits, V, INT4VH_ROWS_F32, draft_ids, draft_probs, uniforms, R, T, V, rules, top_k,
                              temperature, logits_max, argmax_ids, topk_ids, topk_logits, lse, p_draft, n_accepted,
                              rest, logit_rules_verify_workspace_bytes(R, T, V, top_k), stream);
}

} // extern "C"
