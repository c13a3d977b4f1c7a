// logits_common.h -- the rules on logits (penalties, biases, grammar masks) as
// the kernels that read a row of them share it: a wave's walk over its part of
// a row, and the host's checks and shapes (not part of the C ABI).
#ifndef INT4VH_LOGITS_COMMON_H
#define INT4VH_LOGITS_COMMON_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "int4vh.h"
#include "int4vh_internal.h"
#include "int4vh_logits.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace int4vh_detail {

typedef unsigned long long u64;

constexpr int kChunk = 1024;              // tokens of a row that a wave holds at a time
constexpr int kPer = kChunk / 64;         // tokens per lane, 64 apart
constexpr int kMaxWaves = 8;
constexpr int kMaxSlice = kMaxWaves * kChunk;   // tokens of a workgroup's slice
constexpr int kMaxRows = 4096;
constexpr float kNegInf = -__builtin_huge_valf();

// A token's word in LDS: times generated, whether it is in the prompt, and the
// number of its last bias entry (from 1; 0: none).  Where a call's histories
// and biases are short enough all three share 32 bits, which halves the LDS of
// a slice (three workgroups a compute unit instead of two); otherwise entries
// have words of their own.
struct WordLayout {
    uint32_t count, seen;     // bits
    int entry_shift;          // of the entry in a shared word; 0: not shared
};
constexpr WordLayout kShared = {(1u << 20) - 1u, 1u << 20, 21};
constexpr WordLayout kApart = {0x7FFFFFFFu, 0x80000000u, 0};
constexpr long long kSharedHistory = (1ll << 20) - 32;   // generated tokens, drafts on top
constexpr long long kSharedEntries = (1 << 11) - 1;
constexpr long long kMaxHistory = (1ll << 31) - 1 - INT4VH_MAX_T, kMaxEntries = (1ll << 31) - 1;   // kApart's

struct RulesArgs {
    const void *logits;
    long long logits_stride;
    const int32_t *draft;      // [R, T-1] or null
    int R, T, V;
    int4vh_logit_rules r;      // zeros for none
    int has_penalty, has_bias;
    WordLayout word;
    int row_group;             // rows per workgroup
    int ways;                  // waves per row
    int slice;                 // tokens per workgroup: a multiple of ways * kChunk
    int n_lists;               // waves that share a row
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
__device__ __forceinline__ float word_value(uint32_t u)
{
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ float key_value(u64 k)
{
    return word_value((uint32_t)(k >> 32));
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

__device__ __forceinline__ u64 readlane64(u64 k, int src)
{
    return (u64)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(k >> 32), src) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)k, src);
}

// The number of lanes of m below this one.
__device__ __forceinline__ int lane_rank(u64 m)
{
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// A word th (at least 1) that at least k lanes' words reach, and where it can
// be no more than k + 8; 1 where fewer than k lanes have a word, since then
// lower values of the same lanes are wanted too.  Two bits at a time are set
// from the top while enough lanes still reach the word.
__device__ __forceinline__ uint32_t reach_threshold(uint32_t word, int k)
{
    uint32_t th = 0u;
    if (__popcll(__ballot(word != 0u)) < k)
        return 1u;
#pragma nounroll
    for (int shift = 30; shift >= 0; shift -= 2) {
        const int c1 = __popcll(__ballot(word >= (th | 1u << shift)));
        const int c2 = __popcll(__ballot(word >= (th | 2u << shift)));
        const int c3 = __popcll(__ballot(word >= (th | 3u << shift)));
        const uint32_t bits = c3 >= k ? 3u : c2 >= k ? 2u : c1 >= k ? 1u : 0u;
        const int c = c3 >= k ? c3 : c2 >= k ? c2 : c1;
        th |= bits << shift;
        if (bits && c <= k + 8)
            break;
    }
    return th ? th : 1u;
}

// Logit `token` of a row.
template <int kDtype>
__device__ __forceinline__ float load_logit(const void *row, int token)
{
    if constexpr (kDtype == INT4VH_ROWS_F32)
        return static_cast<const float *>(row)[token];
    else
        return from_bits16(static_cast<const uint16_t *>(row)[token], kDtype);
}

template <int kDtype>
__device__ __forceinline__ void store_logit(void *row, int token, float v)
{
    if constexpr (kDtype == INT4VH_ROWS_F32)
        static_cast<float *>(row)[token] = v;
    else
        static_cast<uint16_t *>(row)[token] = (uint16_t)to_bits16(v, kDtype);
}

__device__ __forceinline__ long long clamp64(long long v, long long lo, long long hi)
{
    return v < lo ? lo : v > hi ? hi : v;
}

// A request's part of the histories (generated from `made` on) and of the bias
// entries.
struct Spans {
    long long hb, he, made, bb, be;
};
__device__ __forceinline__ Spans load_spans(const RulesArgs &a, int req)
{
    Spans s = {0, 0, 0, 0, 0};
    if (a.has_penalty && a.r.history) {
        const long long b = a.r.history_offsets[req], e = a.r.history_offsets[req + 1];
        const int prompt = a.r.n_prompt ? a.r.n_prompt[req] : 0;
        s.hb = clamp64(b, 0, a.r.n_history);
        s.he = clamp64(e, 0, a.r.n_history);
        s.made = s.hb + prompt;
    }
    if (a.has_bias) {
        const long long b = a.r.bias_offsets[req], e = a.r.bias_offsets[req + 1];
        s.bb = clamp64(b, 0, a.r.n_bias);
        s.be = clamp64(e, 0, a.r.n_bias);
    }
    return s;
}

// The slice's tokens in one request's history and biases: the words of tokens
// base .. base + S - 1, and the entries' where they lie apart.  Called by the
// whole workgroup, which waits at the end.
__device__ __forceinline__ void prepare_slice(const RulesArgs &a, const Spans &span, int base, int S, uint32_t *words,
                                              uint32_t *entries)
{
    const int tid = threadIdx.x, nt = blockDim.x;
    const long long hb = span.hb, he = span.he, made = span.made, bb = span.bb, be = span.be;
    // Four tokens a load, kFly loads in flight per thread; loads past the end
    // take the last four tokens instead, whose earlier ones are not theirs.
    constexpr int kFly = 4;
    const bool few = he - hb < 4;
    Words4 v[kFly];
    auto load = [&](long long i0) {
        if (few)
            return;
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
            const long long i = i0 + 4ll * u * nt;
            v[u] = *reinterpret_cast<const Words4 *>(a.r.history + (i < he - 4 ? i : he - 4));
        }
    };
    load(hb + 4 * tid);
    int32_t id = -1;
    if (bb + tid < be)
        id = a.r.bias_ids[bb + tid];
    const int n_words = entries == words ? S : 2 * S;
    uint4 *clear = reinterpret_cast<uint4 *>(words);
    for (int i = tid; i < n_words / 4; i += nt)
        clear[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    if (a.has_bias) {
        for (long long i = bb + tid; i < be; i += nt) {
            if (i != bb + tid)
                id = a.r.bias_ids[i];
            const uint32_t at = (uint32_t)id - (uint32_t)base;
            if (id >= 0 && at < (uint32_t)S)
                atomicMax(&entries[at], ((uint32_t)(i - bb) + 1u) << a.word.entry_shift);
        }
        if (entries == words)
            __syncthreads();                  // the maxima are taken before anything is added to them
    }
    auto count = [&](int32_t token, bool prompt) {
        const uint32_t at = (uint32_t)token - (uint32_t)base;
        if (token >= 0 && at < (uint32_t)S) {
            if (prompt)
                atomicOr(&words[at], a.word.seen);
            else
                atomicAdd(&words[at], 1u);
        }
    };
    if (few) {
        if (hb + tid < he)
            count(a.r.history[hb + tid], hb + tid < made);
    } else {
        for (long long i0 = hb + 4 * tid; i0 < he; i0 += 4ll * nt * kFly) {
            if (i0 != hb + 4 * tid)
                load(i0);
#pragma unroll
            for (int u = 0; u < kFly; ++u) {
                const long long i = i0 + 4ll * u * nt, from = i < he - 4 ? i : he - 4;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (from + j >= i)
                        count((int32_t)v[u].w[j], from + j < made);
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float penalise(float l, uint32_t count, float rep, float freq, float pres)
{
    const float x = l > 0.0f ? l / rep : l * rep;
    // tokens of the prompt alone keep x, whatever the other two are (an
    // infinite frequency times a count of 0 would be NaN)
    return count ? x - freq * (float)count - pres : x;
}

// A wave's walk over its part of a slice.  In a grid of (slices of the
// vocabulary, requests, row groups) wave w of a workgroup takes row w / ways of
// the group and the (w % ways)-th part of the slice.
template <int kDtype>
struct SliceWalk {
    static constexpr size_t kSize = kDtype == INT4VH_ROWS_F32 ? 4 : 2;
    // A chunk's logits, and its mask in the lanes below 32, a word each.
    // Tokens past V load the row's last one and are struck out below.
    struct Held {
        float x[kPer];
        uint32_t bits;
    };
    const RulesArgs &a;
    int lane, way;
    int base, begin, n_chunks;                // the slice's first token; this wave's tokens and chunks of them
    int req, t, row;
    int d;                                    // the row's own draft, -1 for none
    uint32_t *words, *entries;
    const char *lrow;
    const uint32_t *mask;
    bool none;                                // nothing is allowed
    int mask_words;
    float rep, freq, pres;
    const float *bias;
    int mine;                                 // lane j holds draft j, for the rows behind it
    Held ha, hb;

    __device__ __forceinline__ void load_x(int c, Held &h) const
    {
        const uint32_t last = (uint32_t)(a.V - 1) * (uint32_t)kSize;
        const int t0 = begin + min(c, n_chunks - 1) * kChunk;
        const uint32_t at = (uint32_t)(t0 + lane) * (uint32_t)kSize;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            h.x[i] = load_logit<kDtype>(lrow + min(at + (uint32_t)(64 * kSize) * i, last), 0);
    }
    __device__ __forceinline__ void load_bits(int c, Held &h) const
    {
        if (mask)
            h.bits = mask[min(((begin + min(c, n_chunks - 1) * kChunk) >> 5) + (lane & 31), mask_words - 1)];
    }
    __device__ __forceinline__ void load(int c, Held &h) const
    {
        load_x(c, h);
        load_bits(c, h);
    }

    // This wave's place in the grid.
    __device__ __forceinline__ SliceWalk(const RulesArgs &args, uint32_t *s_mem)
        : SliceWalk(args, s_mem, blockIdx.x * args.slice, args.slice, blockIdx.y,
                    blockIdx.z * args.row_group + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / args.ways,
                    __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % args.ways, args.ways)
    {
    }

    // Part way_at of n_ways of the S tokens from `first` on, in row t_at of
    // request req_at.  s_mem: the slice's words, then its entries where they lie
    // apart.  The whole workgroup counts the slice, while each wave's chunk
    // `begins` is on its way.
    __device__ __forceinline__ SliceWalk(const RulesArgs &args, uint32_t *s_mem, int first, int S, int req_at,
                                         int t_at, int way_at, int n_ways, int begins = 0)
        : a(args)
    {
        lane = threadIdx.x & 63;
        const int V = a.V;
        words = s_mem;
        entries = s_mem + (a.has_penalty && a.has_bias && !a.word.entry_shift ? S : 0);
        base = first;
        req = req_at;
        t = t_at;
        way = way_at;
        const int part = S / n_ways;
        begin = base + way * part;
        n_chunks = begin < V ? (min(part, V - begin) + kChunk - 1) / kChunk : 0;
        row = req * a.T + min(t, a.T - 1);
        lrow = static_cast<const char *>(a.logits) + (size_t)row * a.logits_stride * kSize;
        ha.bits = hb.bits = 0u;
        if (n_chunks > 0)
            load_x(begins, ha);               // on its way while the slice is counted
        const Spans span = load_spans(a, req);
        mask = nullptr;
        none = false;
        if (a.r.mask) {
            const long long mi = a.r.mask_index ? a.r.mask_index[row] : row;
            none = mi >= a.r.n_masks;
            if (mi >= 0 && !none)
                mask = a.r.mask + (size_t)mi * a.r.mask_stride;
        }
        mask_words = (V + 31) / 32;
        if (n_chunks > 0)
            load_bits(begins, ha);
        if (a.has_penalty || a.has_bias)
            prepare_slice(a, span, base, S, words, entries);
        bias = a.has_bias ? a.r.bias_values + span.bb : nullptr;
    }

    // Whether this wave has a row; no barrier may follow where it has none.
    __device__ __forceinline__ bool live() const
    {
        return t < a.T && t < (int)(blockIdx.z + 1) * a.row_group;
    }

    __device__ __forceinline__ void load_request()
    {
        rep = a.r.repetition ? a.r.repetition[req] : 1.0f;
        freq = a.r.frequency ? a.r.frequency[req] : 0.0f;
        pres = a.r.presence ? a.r.presence[req] : 0.0f;
        mine = -1;
        d = -1;
        if (a.T > 1) {
            const int32_t *dr = a.draft + (size_t)req * (a.T - 1);
            mine = lane < t ? dr[lane] : -1;
            d = t < a.T - 1 ? dr[t] : -1;
        }
    }

    // The rules on the chunk of tokens from chunk0 on; lane l holds tokens
    // chunk0 + l, chunk0 + 64 + l, ...; those past V become -infinity.
    __device__ __forceinline__ void rule(int chunk0, Held &held) const
    {
        float (&x)[kPer] = held.x;
        const int at0 = chunk0 - base + lane;
        if (a.has_penalty || a.has_bias) {
            uint32_t w[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                w[i] = words[at0 + 64 * i];
            if (a.has_penalty) {
                // the drafts in front of this row that lie in the chunk
                for (u64 m = __ballot(mine >= 0 && (uint32_t)(mine - chunk0) < (uint32_t)kChunk); m; m &= m - 1) {
                    const int at = __builtin_amdgcn_readlane(mine, __builtin_ctzll(m)) - chunk0 - lane;
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        w[i] += at == 64 * i ? 1u : 0u;
                }
            }
            const uint32_t known = a.has_penalty ? a.word.count | a.word.seen : 0u;
            const bool here = a.has_bias && entries == words;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (__ballot(w[i] != 0u)) {   // few groups of 64 tokens have any
                    if (w[i] & known)
                        x[i] = penalise(x[i], w[i] & a.word.count, rep, freq, pres);
                    const uint32_t e = here ? w[i] >> a.word.entry_shift : 0u;
                    if (e)
                        x[i] = x[i] + bias[e - 1u];
                }
        }
        if (a.has_bias && entries != words) {
            uint32_t e[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                e[i] = entries[at0 + 64 * i];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (e[i])
                    x[i] = x[i] + bias[e[i] - 1u];
        }
        if (mask || none) {
            const uint32_t bits = none ? 0u : held.bits;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const u64 allowed = (u64)__builtin_amdgcn_readlane(bits, 2 * i + 1) << 32 |
                                    (uint32_t)__builtin_amdgcn_readlane(bits, 2 * i);
                x[i] = __builtin_amdgcn_inverse_ballot_w64(allowed) ? x[i] : kNegInf;
            }
        }
        if (chunk0 + kChunk > a.V)
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                x[i] = chunk0 + 64 * i + lane < a.V ? x[i] : kNegInf;
    }

    // use(chunk0, x) for every chunk of the wave, the next one's loads in flight.
    template <class Use>
    __device__ __forceinline__ void run(Use &&use)
    {
        for (int c = 0; c < n_chunks; c += 2) {
            load(c + 1, hb);
            rule(begin + c * kChunk, ha);
            use(begin + c * kChunk, ha.x);
            if (c + 1 < n_chunks) {
                load(c + 2, ha);
                rule(begin + (c + 1) * kChunk, hb);
                use(begin + (c + 1) * kChunk, hb.x);
            }
        }
    }

    // The same for the chunks of a mask, not 0, whose lowest is the one that the
    // walk begins with.
    template <class Use>
    __device__ __forceinline__ void run_some(uint32_t chunks, Use &&use)
    {
        while (true) {
            int c = __builtin_ctz(chunks);
            chunks &= chunks - 1u;
            if (chunks)
                load(__builtin_ctz(chunks), hb);
            rule(begin + c * kChunk, ha);
            use(begin + c * kChunk, ha.x);
            if (!chunks)
                break;
            c = __builtin_ctz(chunks);
            chunks &= chunks - 1u;
            if (chunks)
                load(__builtin_ctz(chunks), ha);
            rule(begin + c * kChunk, hb);
            use(begin + c * kChunk, hb.x);
            if (!chunks)
                break;
        }
    }
};

// ---------------------------------------------------------------- host side

inline size_t round256(size_t n)
{
    return (n + 255) / 256 * 256;
}

inline bool sizes_ok(int R, int T, int V)
{
    return R >= 1 && T >= 1 && T <= INT4VH_MAX_T && V >= 1 && (long long)R * T <= kMaxRows;
}

constexpr int kMaxV = 1 << 24;

inline int check_rules(const void *logits, int64_t stride, int dtype, const int32_t *draft, int R, int T, int V,
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
    if (r && (r->n_history > kMaxHistory || r->n_bias > kMaxEntries))
        return INT4VH_EUNSUPPORTED;
    return V > kMaxV ? INT4VH_EUNSUPPORTED : INT4VH_OK;
}

inline void fill_rules(RulesArgs &a, const int4vh_logit_rules *r, int T)
{
    a.r = r ? *r : int4vh_logit_rules{};
    const bool any = a.r.repetition || a.r.frequency || a.r.presence;
    a.has_penalty = any && (a.r.history || T > 1);
    a.has_bias = a.r.bias_ids != nullptr;
    // words are shared where both are there; alone, either has the plain ones
    a.word = a.has_penalty && a.has_bias && a.r.n_history <= kSharedHistory && a.r.n_bias <= kSharedEntries ? kShared
                                                                                                         : kApart;
}

struct Shape {
    dim3 grid, block;
    size_t lds;
};

// Slices as long as kMaxSlice spread the counting and a wave's threshold over
// many tokens; shorter ones where there would be fewer than two workgroups a
// compute unit (151936 logits, top-16: 16 requests x 4 rows 29.8 us against
// 34.3 with a target of half a workgroup a unit, 4 x 4 17.3 against 20.5, one
// request's 16 rows 25.3 against 27.7).  A wave has kChunk tokens of a row at
// least.
inline Shape shape_for(RulesArgs &a, size_t wave_bytes, int cus)
{
    const int chunks = (a.V + kChunk - 1) / kChunk;
    a.row_group = a.T < kMaxWaves ? a.T : kMaxWaves;
    a.ways = kMaxWaves / a.row_group;
    while (a.ways > chunks)
        --a.ways;
    const int groups = (a.T + a.row_group - 1) / a.row_group;
    int per = kMaxWaves / a.ways;             // chunks per wave
    while (per > 1 && (long long)((chunks + per * a.ways - 1) / (per * a.ways)) * a.R * groups < 2ll * cus)
        per /= 2;
    while (per > 1 && (per / 2) * a.ways >= chunks)
        per /= 2;                             // no longer than the vocabulary
    a.slice = per * a.ways * kChunk;
    const int slices = (a.V + a.slice - 1) / a.slice;
    a.n_lists = slices * a.ways;
    const int waves = a.row_group * a.ways;
    Shape s;
    s.grid = dim3(slices, a.R, groups);
    s.block = dim3(64 * waves);
    const int arrays = a.word.entry_shift ? 1 : (a.has_penalty ? 1 : 0) + (a.has_bias ? 1 : 0);
    s.lds = (size_t)a.slice * 4 * arrays + waves * wave_bytes;
    return s;
}

inline int current_cus(int *cus)
{
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e, "hipGetDevice");
    *cus = cu_count(dev);
    return INT4VH_OK;
}

} // namespace int4vh_detail

#endif // INT4VH_LOGITS_COMMON_H
