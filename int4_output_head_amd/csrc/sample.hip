// sample.hip -- tokens drawn from logits by given uniform numbers, for MI355X
// (gfx950); definitions in int4vh_sample.h.
//
// Three kernels.  sample_scan_kernel walks the rows as the verification under
// rules does (SliceWalk: the logits are read once, under their rules) and
// leaves of each chunk of 1024 tokens the largest value, and where a setting
// asks for it the sum of the masses, or a value that several of its tokens
// reach.  With no filter a token is drawn from these, and from one chunk that is
// read again.  Otherwise they bound what can be kept: under min_p, nothing more
// than temperature * ln(1 / min_p) below the largest value; under top_p, nothing
// more than temperature * ln(V / ((1 - top_p) * mass of the row)) below, because
// all tokens behind it together would have less than 1 - top_p of that; under top_k,
// nothing below a value that top_k tokens reach.  sample_collect_kernel reads the
// chunks whose largest value passes, a few of them as a rule, and puts what
// passes side by side; sample_draw_kernel, a workgroup per row, finds the
// borders of top_k and top_p among that by histograms of counts and masses, and
// the token by one over tokens.
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>

#include "int4vh.h"
#include "int4vh_internal.h"
#include "int4vh_sample.h"
#include "logits_common.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace {

using namespace int4vh_detail;

constexpr int kDrawThreads = 1024;
constexpr int kFew = 512;                 // candidates that are compared with each other
constexpr int kMany = 4096;               // candidates worth a pass that leaves fewer of them
constexpr int kBins = kDrawThreads;

// Words between counters that workgroups of all XCDs add to: a cache line each
// (side by side, 256 rows' collection took 100 us instead of 30).
constexpr int kPad = 32;

struct SampleArgs : RulesArgs {
    int4vh_sampling s;
    const float *uniforms;     // [R*T]
    const float *accept;       // [R, T-1] or null
    int bits;                  // masses are multiples of 2^-bits
    float *tops;               // [R*T, chunks] largest value
    float *bars;               // [R*T, chunks] value that each() of the chunk's tokens reach, under top_k
    float *refs;               // [R*T, chunks] largest value, less the row's draft where drafts are verified,
    double *sums;              // [R*T, chunks] and the masses' sum relative to it, likewise
    u64 *cand;                 // [R*T, V] candidates' keys, in any order,
    int *counts;               // [R*T][kPad] their number
    float *lows;               // [R*T] and a value that all of them reach
    float *draft_logit;        // [R*T] ruled logit of the row's draft, where it is in [0, V)
    uint32_t *tickets;         // [R] rows done
    uint32_t *oks;             // [R*T] whether the row's draft is accepted
    int32_t *token_ids;
    float *token_probs, *p_draft;
    int32_t *n_accepted;
};

constexpr int kGroups = 4;                    // groups of chunks per lane in lowest_kept

// A request's settings: k = 0, p = 1 and mp = 0 keep all.
struct Settings {
    double inv_t;                             // log2(e) / temperature
    float t;
    int k;
    float p, mp;
    __device__ __forceinline__ bool filtered() const { return k > 0 || p < 1.0f || mp > 0.0f; }
    // whether the sums of the chunks are wanted
    __device__ __forceinline__ bool summed() const { return k == 0 && (p < 1.0f || mp <= 0.0f); }
    // under top_k: tokens of each of n chunks, so that some of the chunks, and no more
    // than lowest_kept has groups for, have top_k of them (600000 tokens, top-k 257: 34 us;
    // of one token a chunk, which took 257 chunks and so had no bound, 2394)
    __device__ __forceinline__ int each(int n) const
    {
        int j = 1;
        while (j < 64 && ((long long)j * n < 2ll * k || j * 64 * kGroups < k))
            j *= 2;
        return j;
    }
};
__device__ __forceinline__ Settings load_settings(const SampleArgs &a, int req)
{
    Settings s;
    s.t = a.s.temperatures ? a.s.temperatures[req] : a.s.temperature;
    s.k = a.s.top_ks ? a.s.top_ks[req] : a.s.top_k;
    s.p = a.s.top_ps ? a.s.top_ps[req] : a.s.top_p;
    s.mp = a.s.min_ps ? a.s.min_ps[req] : a.s.min_p;
    s.k = s.k <= 0 || s.k >= a.V ? 0 : s.k;
    s.p = s.p < 1.0f ? fmaxf(s.p, 0.0f) : 1.0f;
    s.mp = s.mp > 0.0f ? fminf(s.mp, 1.0f) : 0.0f;
    if (!(s.t > 0.0f && s.t < __builtin_huge_valf())) {
        s.t = 0.0f;
        s.k = 1;
        s.p = 1.0f;
        s.mp = 0.0f;
    }
    s.inv_t = s.t > 0.0f ? 1.4426950408889634 / (double)s.t : 0.0;
    return s;
}

// 2^z for z <= 0 (NaN and values below -1000 count as -1000), of relative error
// 2^-40: the whole part of z goes into the exponent, the rest, |f| <= 1/2, through
// the polynomial of degree 8 whose largest relative error is least (7.8e-13, by
// exchange of its extrema).
__device__ __forceinline__ double exp2_below(double z)
{
    z = fmax(z, -1000.0);
    const double t = z + 0x1.8p52, f = z - (t - 0x1.8p52);     // t holds the whole part in its low word
    double p = 1.3175858136257845e-06;
    p = __builtin_fma(p, f, 1.5309737421323303e-05);
    p = __builtin_fma(p, f, 1.540385174860361e-04);
    p = __builtin_fma(p, f, 1.3333452062251618e-03);
    p = __builtin_fma(p, f, 9.618128542862621e-03);
    p = __builtin_fma(p, f, 5.550410939341707e-02);
    p = __builtin_fma(p, f, 2.4022650698880368e-01);
    p = __builtin_fma(p, f, 6.931471805465141e-01);
    p = __builtin_fma(p, f, 9.999999999997623e-01);
    return __hiloint2double(__double2hiint(p) + (__double2loint(t) << 20), __double2loint(p));
}

// The mass of a value x at most m, relative to that of m; 1 at m itself, so that
// infinities do not meet, and 0 for -infinity and NaN.
__device__ __forceinline__ double mass_below(float x, float m, double inv_t)
{
    return x == m ? 1.0 : x > kNegInf ? exp2_below(((double)x - (double)m) * inv_t) : 0.0;
}

// How far below a row's largest value m a kept token may lie, with slack for the
// roundings of this bound; the row has at least the mass `mass` relative to m.
// Infinite where the settings do not bound it, and 0 below an infinite m, as long
// as they do.
__device__ __forceinline__ float reach_of(const Settings &set, int V, float m, float mass)
{
    float reach = __builtin_huge_valf();
    if (set.t == 0.0f)
        return 0.0f;
    if (set.mp > 0.0f && (set.k == 0 || set.p >= 1.0f))
        reach = -set.t * logf(set.mp);
    if (set.p < 1.0f && set.k == 0)
        reach = fminf(reach, set.t * logf((float)V / ((1.0f - set.p) * mass)));
    if (reach == __builtin_huge_valf())
        return reach;
    return m == __builtin_huge_valf() ? 0.0f : reach * (1.0f + 0x1p-18f) + set.t * 0x1p-18f + fabsf(m) * 0x1p-20f;
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
}

// Bound by memory where no sums are wanted (256 x 151936 in binary32, 156 MB: 27
// us, 5.8 TB/s with part of it in the last-level cache), else by the masses in
// binary64, some 20 instructions each (41 us).
template <int kDtype>
__global__ void __launch_bounds__(64 * kMaxWaves) sample_scan_kernel(SampleArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint32_t s_mem[];
    SliceWalk<kDtype> walk(a, s_mem);
    if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x < a.T) {
        a.counts[(blockIdx.y * a.T + threadIdx.x) * kPad] = 0;
        if (threadIdx.x == 0)
            a.tickets[blockIdx.y] = 0u;
    }
    if (!walk.live())
        return;                               // no barrier follows
    walk.load_request();
    const int lane = walk.lane, row = walk.row, d = walk.d, V = a.V;
    const Settings set = load_settings(a, walk.req);
    const bool summed = set.summed();
    const int n_chunks = (V + kChunk - 1) / kChunk, each = set.k > 0 ? set.each(n_chunks) : 1;
    walk.run([&](int chunk0, float (&x)[kPer]) {
        const size_t at = (size_t)row * n_chunks + chunk0 / kChunk;
        float best = kNegInf;                 // fmaxf passes over NaN
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            best = fmaxf(best, x[i]);
        float m = wave_max(best);
        if (lane == 0)
            a.tops[at] = m;
        if (each > 1) {
            const uint32_t th = reach_threshold(best > kNegInf ? order_word(best) : 0u, each);
            if (lane == 0)
                a.bars[at] = th > 1u ? word_value(th) : kNegInf;
        }
        const uint32_t da = (uint32_t)d - (uint32_t)chunk0;
        if (d >= 0 && d < V && da < (uint32_t)kChunk) {
            float v = kNegInf;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const bool own = (int)(da >> 6) == i && (int)(da & 63u) == lane;
                v = own ? x[i] : v;
                if (a.accept && own)
                    x[i] = kNegInf;           // apart from the sums
            }
            if ((int)(da & 63u) == lane)
                a.draft_logit[row] = v;
            best = kNegInf;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                best = fmaxf(best, x[i]);
            m = wave_max(best);
        }
        if (summed) {
            double s = 0.0;
            if (fabsf(m) < __builtin_huge_valf()) {
                // -infinity and NaN come out as 2^-1000
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    s += exp2_below(((double)x[i] - (double)m) * set.inv_t);
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    s += x[i] == m ? 1.0 : 0.0;
            }
            s = wave_sum_f64(s);
            if (lane == 0) {
                a.refs[at] = m;
                a.sums[at] = m > kNegInf ? s : 0.0;
            }
        }
    });
}

// The row's largest value, and one that nothing that is kept lies below, from
// what the scan has left of its chunks.  A whole wave.  A top_k of more than 64 tokens
// a chunk, or of more than 16384, has no such value: all of the row are candidates then,
// and draw_many finds the border (151936 tokens, top-k 9500 81 us, 9600 632).
__device__ __forceinline__ float lowest_kept(const SampleArgs &a, const Settings &set, int row, int lane, float &gm)
{
    const int n = (a.V + kChunk - 1) / kChunk, each = set.k > 0 ? set.each(n) : 1;
    const float *tops = a.tops + (size_t)row * n, *bars = each > 1 ? a.bars + (size_t)row * n : tops;
    float most[kGroups], m = kNegInf;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
        most[g] = kNegInf;
    for (int c0 = 0; c0 < n; c0 += 64 * kGroups)
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            if (c0 + 64 * g + lane < n) {
                m = fmaxf(m, tops[c0 + 64 * g + lane]);
                most[g] = fmaxf(most[g], bars[c0 + 64 * g + lane]);
            }
    gm = wave_max(m);
    float mass = 1.0f;
    if (set.p < 1.0f && set.k == 0 && fabsf(gm) < __builtin_huge_valf()) {
        // (without a draft that is apart: at least this)
        const float *refs = a.refs + (size_t)row * n;
        const double *sums = a.sums + (size_t)row * n;
        float s = 0.0f;
        for (int c = lane; c < n; c += 64)
            s += refs[c] > kNegInf ? (float)sums[c] * exp2f((refs[c] - gm) * (float)set.inv_t) : 0.0f;
        mass = fmaxf(mass, wave_sum(s) * (1.0f - 0x1p-10f));
    }
    float low = gm - reach_of(set, a.V, gm, mass);  // (NaN: no bound)
    low = fmaxf(low, -3.402823466e38f);
    const int want = set.k > 0 ? (set.k + each - 1) / each : 0;
    if (set.k == 1)
        low = fmaxf(gm, -3.402823466e38f);    // not -infinity, which all of a row without a token has
    else if (want > 0 && want <= n && want <= 64 * kGroups) {
        // a word that at least `want` groups reach, two bits at a time
        uint32_t word[kGroups], th = 0u;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            word[g] = most[g] > kNegInf ? order_word(most[g]) : 0u;
        auto reach = [&](uint32_t w) {
            int c = 0;
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                c += __popcll(__ballot(word[g] >= w));
            return c;
        };
        if (reach(1u) >= want) {
#pragma nounroll
            for (int shift = 30; shift >= 0; shift -= 2) {
                const uint32_t bits = reach(th | 3u << shift) >= want   ? 3u
                                      : reach(th | 2u << shift) >= want ? 2u
                                      : reach(th | 1u << shift) >= want ? 1u
                                                                        : 0u;
                th |= bits << shift;
                if (bits && reach(th) <= want + 8)
                    break;
            }
            low = fmaxf(low, word_value(th));
        }
    }
    return low;
}

// Grid and workgroups of the scan; chunks whose largest value is too low are not
// read again.  256 x 151936: 9 us for the best token alone, 21 under top-k 20, 36
// under top-p 0.5, 52 where nearly all chunks pass (temperature 1.3 under top-p
// 0.95); one row 6 to 13 us, a chain of latencies: the bound, the rules' counts,
// the logits, the counter.
template <int kDtype>
__global__ void __launch_bounds__(64 * kMaxWaves) sample_collect_kernel(SampleArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint32_t s_mem[];
    __shared__ int s_any;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int req = blockIdx.y, t = blockIdx.z * a.row_group + wave / a.ways, way = wave % a.ways;
    const Settings set = load_settings(a, req);
    if (!set.filtered())
        return;
    if (threadIdx.x == 0)
        s_any = 0;
    __syncthreads();
    const bool live = t < a.T && t < (int)(blockIdx.z + 1) * a.row_group;
    const int V = a.V, n_chunks = (V + kChunk - 1) / kChunk, row = req * a.T + t;
    const int part = a.slice / a.ways / kChunk, c0 = blockIdx.x * (a.slice / kChunk) + way * part;
    float gm = kNegInf, low = kNegInf;
    uint32_t chunks = 0u;
    if (live) {
        low = lowest_kept(a, set, row, lane, gm);
        const bool more = lane < part && c0 + lane < n_chunks && a.tops[(size_t)row * n_chunks + c0 + lane] >= low;
        chunks = (uint32_t)__ballot(more);
        if (chunks && lane == 0)
            s_any = 1;
        if (blockIdx.x == 0 && way == 0 && lane == 0)
            a.lows[row] = low;
    }
    __syncthreads();
    if (!s_any)
        return;
    SliceWalk<kDtype> walk(a, s_mem, blockIdx.x * a.slice, a.slice, req, t, way, a.ways,
                           chunks ? __builtin_ctz(chunks) : 0);
    if (!chunks)
        return;                               // no barrier follows
    walk.load_request();
    u64 *cand = a.cand + (size_t)row * V;
    walk.run_some(chunks, [&](int chunk0, float (&x)[kPer]) {
        u64 m[kPer];
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            m[i] = __ballot(x[i] >= low);
            n += __popcll(m[i]);
        }
        int at = 0;
        if (lane == 0)
            at = atomicAdd(&a.counts[row * kPad], n);
        at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (m[i]) {
                if (x[i] >= low)
                    cand[at + lane_rank(m[i])] = order_key(x[i], chunk0 + 64 * i + lane);
                at += __popcll(m[i]);
            }
    });
}

// ---------------------------------------------------------------- drawing

// Reductions and scans over the workgroup; all threads, `s` of 16 values per
// use, free again after the next barrier.
__device__ __forceinline__ float block_max(float v, float *s)
{
    v = wave_max(v);
    if ((threadIdx.x & 63) == 0)
        s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[threadIdx.x & 15];
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1)
        v = fmaxf(v, __shfl_xor(v, off));
    __syncthreads();
    return v;
}

__device__ __forceinline__ u64 shfl_up64(u64 v, int off)
{
    const uint32_t lo = __shfl_up((uint32_t)v, off), hi = __shfl_up((uint32_t)(v >> 32), off);
    return ((u64)hi << 32) | lo;
}

// The inclusive sum over the threads up to this one, and the whole sum.
__device__ __forceinline__ u64 block_scan(u64 v, u64 *s, u64 &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const u64 o = shfl_up64(v, off);
        v += lane >= off ? o : 0ull;
    }
    if (lane == 63)
        s[wave] = v;
    __syncthreads();
    u64 before = 0ull;
    total = 0ull;
#pragma unroll
    for (int w = 0; w < kDrawThreads / 64; ++w) {
        before += w < wave ? s[w] : 0ull;
        total += s[w];
    }
    __syncthreads();
    return v + before;
}

struct DrawLds {
    u64 few[kFew];                            // few candidates that are compared with each other,
    u64 units[kFew];                          // and their masses
    u64 hist[kBins];
    uint32_t hits[kBins];
    __attribute__((aligned(16))) uint32_t words[2 * kChunk];   // the rules' words of one chunk
    u64 scan[16];
    float fl[16];
    u64 found, rest;
    int at, n, some;
    float value;
};

__device__ __forceinline__ u64 fixed(double mass, int bits)
{
    return (u64)llrint(ldexp(mass, bits));
}
// The same for a mass of at most 1 and at most 50 bits: added to 3 * 2^51 the
// number lies, rounded, in the low bits.
__device__ __forceinline__ u64 fixed_one(double mass, int bits)
{
    return (u64)__double_as_longlong(ldexp(mass, bits) + 0x1.8p52) & ((1ull << 51) - 1ull);
}
__device__ __forceinline__ double floating(u64 sum, int bits)
{
    return ldexp((double)sum, -bits);
}

// The sum that a token's has to exceed.
__device__ __forceinline__ u64 drawn(float u, u64 total)
{
    const double y = u > 0.0f ? floor((double)u * (double)total) : 0.0;
    return y < (double)total ? min((u64)y, total - 1ull) : total - 1ull;
}

// Keys by value, then token: 56 bits that are all in use; and by token alone,
// the lowest first.
__device__ __forceinline__ u64 value_key(u64 key)
{
    return (key >> 32) << 24 | (key & 0xFFFFFFull);
}
__device__ __forceinline__ u64 token_key(u64 key)
{
    return key & 0xFFFFFFull;
}

// lds.hist emptied, and no bin found.
__device__ __forceinline__ void clear_bins(DrawLds &lds)
{
    lds.hist[threadIdx.x] = 0ull;
    if (threadIdx.x == 0) {
        lds.at = -1;
        lds.n = 0;
    }
    __syncthreads();
}

// The bin, of lds.hist as the threads have filled it, in which the sum from the
// first on reaches target_of(sum of all) (-1: none does); lds.rest is the sum in
// front of it.
template <class Target>
__device__ __forceinline__ int border_bin(u64 above, DrawLds &lds, Target &&target_of)
{
    __syncthreads();
    u64 total;
    const u64 mine = lds.hist[threadIdx.x], upto = block_scan(mine, lds.scan, total) + above;
    const u64 target = target_of(total);
    if (upto - mine < target && upto >= target) {
        lds.at = threadIdx.x;
        lds.rest = upto - mine;
    }
    __syncthreads();
    return lds.at;
}

// The key (by `order`) of the last candidate whose predecessors, those of
// larger keys, weigh less than `target` (at least 1) together; 0 where all
// candidates weigh less than that.  each(f) calls f with every candidate once;
// keys lie in [lo, hi].
template <class Each, class Order, class Weight>
__device__ __forceinline__ u64 border(Each &&each, u64 lo, u64 hi, u64 target, DrawLds &lds, Order &&order,
                                      Weight &&weight)
{
    u64 above = 0ull;
    const int tid = threadIdx.x;
    while (true) {
        // bins of 2^shift keys, from hi down
        const int width = hi > lo ? 64 - __builtin_clzll(hi - lo) : 1, shift = width > 10 ? width - 10 : 0;
        lds.hits[tid] = 0u;
        clear_bins(lds);
        each([&](u64 key) {
            const u64 o = order(key);
            if (o >= lo && o <= hi) {
                const u64 w = weight(key);
                if (w) {
                    const int bin = (int)((hi - o) >> shift);
                    atomicAdd(&lds.hist[bin], w);
                    atomicAdd(&lds.hits[bin], 1u);
                }
            }
        });
        const int bin = border_bin(above, lds, [&](u64) { return target; });
        if (bin < 0)
            return 0ull;
        above = lds.rest;
        const uint32_t hits = lds.hits[bin];
        hi -= (u64)bin << shift;
        const u64 below = hi - ((1ull << shift) - 1ull);
        lo = below > lo && below <= hi ? below : lo;
        if (hits == 1u)
            break;
        __syncthreads();
    }
    each([&](u64 key) {
        const u64 o = order(key);
        if (o >= lo && o <= hi && weight(key))
            lds.found = o;
    });
    __syncthreads();
    const u64 key = lds.found;
    __syncthreads();
    return key;
}

struct Draw {
    int token;
    float prob, p_draft;
};

// A row's candidates and what they are drawn with.
struct Row {
    const SampleArgs &a;
    const Settings &set;
    float gm;                                 // the largest value
    double whole;                             // mass of the row, where top_p applies to all of it
    int d;                                    // the draft that is left out, or -1
    float u;

    __device__ __forceinline__ double mass(u64 key, float ref) const
    {
        return set.t > 0.0f ? mass_below(key_value(key), ref, set.inv_t) : 1.0;
    }
    __device__ __forceinline__ u64 units(u64 key, float ref) const { return fixed_one(mass(key, ref), a.bits); }
    // what a sum has to reach to hold top_p of `all`; at least 1, for the best token
    __device__ __forceinline__ u64 share(u64 all) const
    {
        const double bar = ceil((double)set.p * (double)all);
        return bar > 1.0 ? (u64)bar : 1ull;
    }
};

// Appends to an array, at most `most` of them, with a count in LDS; the lanes that
// call it.
__device__ __forceinline__ void append(u64 key, u64 *to, int *n, int most)
{
    const u64 m = __ballot(true);
    const int first = __builtin_ctzll(m);
    int at = 0;
    if ((int)(threadIdx.x & 63) == first)
        at = atomicAdd(n, __popcll(m));
    at = __shfl(at, first) + lane_rank(m);
    if (at < most)
        to[at] = key;
}

// A group of threads for each of n <= kFew keys of lds.few, all of which it
// compares with its own: the lead has the results.
struct Ranked {
    int i, rank;                              // rank: the number of larger keys
    bool mine, lead;
    u64 key, before;                          // before: what they weigh
    int group;

    __device__ __forceinline__ Ranked(int n, const DrawLds &lds)
    {
        group = kDrawThreads / kFew;
        while (group < 64 && 2 * group * n <= kDrawThreads)
            group *= 2;
        i = threadIdx.x / group;
        mine = i < n;
        lead = mine && threadIdx.x % group == 0;
        key = mine ? lds.few[i] : 0ull;
    }
    // with the masses in lds.units
    template <class Order>
    __device__ __forceinline__ void rank_by(int n, const DrawLds &lds, Order &&order)
    {
        rank = 0;
        before = 0ull;
        const u64 own = order(key);
        for (int j = threadIdx.x % group; j < n; j += group) {
            const bool more = order(lds.few[j]) > own;
            rank += more;
            before += more ? lds.units[j] : 0ull;
        }
        for (int off = 1; off < group; off <<= 1) {
            rank += __shfl_xor(rank, off);
            before += shfl_xor64(before, off);
        }
    }
};

// The token at which the sum of the masses by token exceeds `target`, less
// `front` that lies before the n keys of lds.few with masses lds.units.
__device__ __forceinline__ void draw_ranked(Ranked &k, int n, u64 w, u64 front, u64 target, double share, DrawLds &lds)
{
    k.rank_by(n, lds, token_key);
    if (k.lead && front + k.before <= target && target < front + k.before + w) {
        lds.at = key_token(k.key);
        lds.value = (float)share;
    }
    __syncthreads();
}

// Few candidates, n <= kFew, in lds.few.
__device__ __forceinline__ Draw draw_few(const Row &r, int n, DrawLds &lds)
{
    __syncthreads();
    Ranked k(n, lds);
    const u64 own = k.mine ? r.units(k.key, r.gm) : 0ull;
    if (k.lead)
        lds.units[k.i] = own;
    if (threadIdx.x == 0)
        lds.some = 0;
    __syncthreads();
    k.rank_by(n, lds, [](u64 key) { return key; });
    bool kept = k.mine && (r.set.k == 0 || k.rank < r.set.k);
    if (r.set.p < 1.0f) {
        u64 all;
        if (r.set.k > 0)
            block_scan(k.lead && kept ? own : 0ull, lds.scan, all);
        else
            all = fixed(r.whole, r.a.bits);
        kept = kept && k.before < r.share(all);
    }
    kept = kept && (r.set.mp <= 0.0f || r.mass(k.key, r.gm) >= (double)r.set.mp);
    Draw out = {-1, 0.0f, 0.0f};
    float ref = r.gm;
    u64 w = kept ? own : 0ull;
    if (r.d >= 0) {
        u64 all;
        block_scan(k.lead ? w : 0ull, lds.scan, all);
        const bool draft = kept && key_token(k.key) == r.d;
        if (draft && k.lead) {
            lds.some = 1;
            lds.value = (float)(r.mass(k.key, r.gm) / floating(all, r.a.bits));
        }
        kept = kept && !draft;
        ref = block_max(kept ? key_value(k.key) : kNegInf, lds.fl);
        out.p_draft = lds.some ? lds.value : 0.0f;
        if (ref == kNegInf)
            return out;
        w = kept ? r.units(k.key, ref) : 0ull;
    }
    u64 total;
    block_scan(k.lead ? w : 0ull, lds.scan, total);
    if (k.lead)
        lds.units[k.i] = w;
    __syncthreads();
    draw_ranked(k, n, w, 0ull, drawn(r.u, total), w ? r.mass(k.key, ref) / floating(total, r.a.bits) : 0.0, lds);
    out.token = lds.at;
    out.prob = lds.value;
    return out;
}

// f with each of the n >= 2 candidates, the next 2 * kFly of each thread in flight.
struct __attribute__((aligned(8))) KeyPair { u64 a, b; };
template <class F>
__device__ __forceinline__ void each_of(const u64 *cand, int n, F &&f)
{
    constexpr int kFly = 4;
    KeyPair next[kFly];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            const int i = i0 + 2 * (j * kDrawThreads + (int)threadIdx.x);
            // (the last pair of an odd number begins one key earlier)
            next[j] = KeyPair{0ull, 0ull};
            if (i < n) {
                next[j] = *reinterpret_cast<const KeyPair *>(cand + min(i, n - 2));
                if (i + 1 == n)
                    next[j] = KeyPair{next[j].b, 0ull};
            }
        }
    };
    load(0);
    for (int i0 = 0; i0 < n; i0 += 2 * kFly * kDrawThreads) {
        KeyPair key[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j)
            key[j] = next[j];
        if (i0 + 2 * kFly * kDrawThreads < n)
            load(i0 + 2 * kFly * kDrawThreads);
        // four copies of f: the keys move down by two pairs
#pragma nounroll
        for (int j = 0; j < kFly && i0 + 2 * j * kDrawThreads < n; j += 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (key[k].a)
                    f(key[k].a);
                if (key[k].b)
                    f(key[k].b);
            }
#pragma unroll
            for (int k = 0; k + 2 < kFly; ++k)
                key[k] = key[k + 2];
        }
    }
}

// Those of the n candidates for which take() holds, in lds.few; their number.
template <class Take>
__device__ __forceinline__ int gather(const u64 *cand, int n, DrawLds &lds, Take &&take)
{
    if (threadIdx.x == 0)
        lds.n = 0;
    __syncthreads();
    each_of(cand, n, [&](u64 key) {
        if (take(key))
            append(key, lds.few, &lds.n, kFew);
    });
    __syncthreads();
    return lds.n;
}

// The last key, by value, of those that take() takes (a bin) whose predecessors
// weigh less than `target` together, those in front of the bin `above`; false
// where these are too many.
template <class Take, class Weight>
__device__ __forceinline__ bool border_among(const u64 *cand, int n, u64 above, u64 target, DrawLds &lds, Take &&take,
                                             Weight &&weight, u64 &least)
{
    const int m = gather(cand, n, lds, take);
    if (m > kFew)
        return false;
    Ranked k(m, lds);
    if (k.lead)
        lds.units[k.i] = weight(k.key);
    if (threadIdx.x == 0)
        lds.found = ~0ull;
    __syncthreads();
    k.rank_by(m, lds, [](u64 key) { return key; });
    if (k.lead && above + k.before < target)
        atomicMin(&lds.found, value_key(k.key));
    __syncthreads();
    least = lds.found;
    __syncthreads();
    return true;
}

// n candidates, from the largest value down to `low`.  False where a bin holds too
// many of them.
__device__ __forceinline__ bool draw_binned(const Row &r, u64 *cand, int n, float low, DrawLds &lds, Draw &out)
{
    const Settings &set = r.set;
    const int tid = threadIdx.x, bits = r.a.bits;
    // bins by the distance from the largest value
    const float gm = r.gm, scale = gm > low && gm - low < __builtin_huge_valf() ? (float)kBins / (gm - low) : 0.0f;
    auto bin_of = [&](u64 key) {
        const float x = key_value(key);
        return x >= gm ? 0 : min((int)((gm - x) * scale), kBins - 1);
    };
    auto units = [&](u64 key) { return r.units(key, gm); };
    // Of many candidates, those down to the border's bin move behind the others, as
    // the row's place has room for V of them: all that follows reads these alone
    // (151936 logits at temperature 1.3 under top-p 0.95, 256 rows of 47000
    // candidates: 78 us instead of 130; below kMany the pass costs what it saves:
    // under top-p 0.5 and 0.95 at temperature 1 24.8 and 29.3 us without, 25.6 and
    // 28.1 with it).  Under top_k and top_p they may move twice: what is left of the
    // row's place counts from where they lie.
    const u64 *const place_end = cand + r.a.V;
    auto narrow = [&](int bin) {
        const int room = (int)(place_end - cand) - n;
        if (bin < 0 || n <= kMany)
            return;
        if (tid == 0)
            lds.n = 0;
        __syncthreads();
        each_of(cand, n, [&](u64 key) {
            if (bin_of(key) <= bin)
                append(key, cand + n, &lds.n, room);
        });
        __syncthreads();
        const int m = lds.n;
        __syncthreads();
        if (m >= 2 && m <= room) {
            cand += n;
            n = m;
        }
    };
    u64 least = 0ull, target = 0ull;
    if (set.k > 0) {
        clear_bins(lds);
        each_of(cand, n, [&](u64 key) { atomicAdd(&lds.hist[bin_of(key)], 1ull); });
        const int bin = border_bin(0ull, lds, [&](u64) { return (u64)set.k; });
        const u64 above = lds.rest;
        __syncthreads();
        narrow(bin);
        if (bin >= 0 && !border_among(cand, n, above, (u64)set.k, lds, [&](u64 key) { return bin_of(key) == bin; },
                                      [](u64) { return 1ull; }, least))
            return false;
    }
    if (set.p < 1.0f) {
        clear_bins(lds);
        each_of(cand, n, [&](u64 key) {
            if (value_key(key) >= least)
                atomicAdd(&lds.hist[bin_of(key)], units(key));
        });
        const int bin = border_bin(0ull, lds, [&](u64 all) {
            return target = r.share(set.k > 0 ? all : fixed(r.whole, bits));
        });
        const u64 above = lds.rest;
        __syncthreads();
        narrow(bin);
        u64 last = 0ull;
        if (bin >= 0 && !border_among(cand, n, above, target, lds,
                                      [&](u64 key) { return bin_of(key) == bin && value_key(key) >= least; }, units,
                                      last))
            return false;
        least = last > least ? last : least;
    }
    auto kept = [&](u64 key) {
        return value_key(key) >= least && (set.mp <= 0.0f || r.mass(key, gm) >= (double)set.mp);
    };
    // by token, the draft's apart: bins of 2^shift neighbours
    const int shift = max(0, 32 - __builtin_clz(r.a.V) - 10);
    float ref = gm;
    auto drawable = [&](u64 key) { return kept(key) && key_token(key) != r.d ? r.units(key, ref) : 0ull; };
    u64 total = 0ull;
    auto token_bin = [&]() {
        return border_bin(0ull, lds, [&](u64 all) {
            total = all;
            return drawn(r.u, all) + 1ull;
        });
    };
    if (tid == 0)
        lds.some = 0;
    clear_bins(lds);
    float v = kNegInf;                        // the largest value beside the draft's
    each_of(cand, n, [&](u64 key) {
        if (kept(key)) {
            if (key_token(key) == r.d) {
                lds.some = 1;
                lds.value = key_value(key);
            } else {
                v = fmaxf(v, key_value(key));
                const u64 w = units(key);
                if (w)
                    atomicAdd(&lds.hist[key_token(key) >> shift], w);
            }
        }
    });
    int bin = token_bin();
    out.p_draft = 0.0f;
    if (r.d >= 0) {
        if (lds.some) {
            const double md = set.t > 0.0f ? mass_below(lds.value, gm, set.inv_t) : 1.0;
            out.p_draft = (float)(md / (md + floating(total, bits)));
        }
        ref = block_max(v, lds.fl);
        if (ref == kNegInf)
            return true;
        if (ref < gm) {
            // the draft was the best token: masses relative to the next one
            clear_bins(lds);
            each_of(cand, n, [&](u64 key) {
                const u64 w = drawable(key);
                if (w)
                    atomicAdd(&lds.hist[key_token(key) >> shift], w);
            });
            bin = token_bin();
        }
    }
    const u64 above = lds.rest;
    __syncthreads();
    const int m = gather(cand, n, lds, [&](u64 key) { return key_token(key) >> shift == bin && kept(key); });
    if (m > kFew)
        return false;
    Ranked k(m, lds);
    const u64 w = k.mine ? drawable(k.key) : 0ull;
    if (k.lead)
        lds.units[k.i] = w;
    __syncthreads();
    draw_ranked(k, m, w, above, drawn(r.u, total), w ? r.mass(k.key, ref) / floating(total, bits) : 0.0, lds);
    out.token = lds.at;
    out.prob = lds.value;
    return true;
}

// Any number of them: the borders by histograms.  each(f): f with every
// candidate once.
template <class Each>
__device__ __forceinline__ Draw draw_many(const Row &r, Each &&each, DrawLds &lds)
{
    const Settings &set = r.set;
    const int tid = threadIdx.x, bits = r.a.bits;
    u64 least = 0ull;
    if (set.k > 0 || set.p < 1.0f) {
        // the smallest value among the candidates
        float v = __builtin_huge_valf();
        each([&](u64 key) { v = fminf(v, key_value(key)); });
        v = -block_max(-v, lds.fl);
        const u64 lo = (u64)order_word(v) << 24, hi = (u64)order_word(r.gm) << 24 | 0xFFFFFFull;
        if (set.k > 0)
            least = border(each, lo, hi, (u64)set.k, lds, value_key, [](u64) { return 1ull; });
        if (set.p < 1.0f) {
            u64 all;
            if (set.k > 0) {
                u64 w = 0ull;
                each([&](u64 key) { w += value_key(key) >= least ? r.units(key, r.gm) : 0ull; });
                block_scan(w, lds.scan, all);
            } else {
                all = fixed(r.whole, bits);
            }
            const u64 last = border(each, lo, hi, r.share(all), lds, value_key,
                                    [&](u64 key) { return r.units(key, r.gm); });
            least = last > least ? last : least;
        }
    }
    auto kept = [&](u64 key) {
        return value_key(key) >= least && (set.mp <= 0.0f || r.mass(key, r.gm) >= (double)set.mp);
    };
    // the draft's share, and the largest value without it
    Draw out = {-1, 0.0f, 0.0f};
    float ref = r.gm;
    if (r.d >= 0) {
        if (tid == 0)
            lds.some = 0;
        float v = kNegInf;
        u64 w = 0ull;
        __syncthreads();
        each([&](u64 key) {
            if (kept(key)) {
                w += r.units(key, r.gm);
                if (key_token(key) == r.d) {
                    lds.some = 1;
                    lds.value = key_value(key);
                } else {
                    v = fmaxf(v, key_value(key));
                }
            }
        });
        u64 all;
        block_scan(w, lds.scan, all);
        if (lds.some)
            out.p_draft = (float)((set.t > 0.0f ? mass_below(lds.value, r.gm, set.inv_t) : 1.0) / floating(all, bits));
        ref = block_max(v, lds.fl);
        if (ref == kNegInf)
            return out;
    }
    auto drawable = [&](u64 key) { return kept(key) && key_token(key) != r.d ? r.units(key, ref) : 0ull; };
    u64 w = 0ull, total;
    each([&](u64 key) { w += drawable(key); });
    block_scan(w, lds.scan, total);
    const u64 at = border(each, 0ull, 0xFFFFFFull, drawn(r.u, total) + 1ull, lds, token_key, drawable);
    each([&](u64 key) {
        if (token_key(key) == at)
            lds.value = (float)(r.mass(key, ref) / floating(total, bits));
    });
    __syncthreads();
    out.token = (int)(0xFFFFFFull - at);
    out.prob = lds.value;
    return out;
}

// A workgroup per row.  256 rows of 151936: 13 to 17 us for up to kFew candidates
// (a row alone 7 to 9, a chain of reductions over the workgroup), 25 to 29 under
// top-p 0.5 and 0.95, 77 for 47000 candidates a row (alone 52: two passes of some
// 60 instructions over all of them on one compute unit, the others on few).
template <int kDtype>
__global__ void __launch_bounds__(kDrawThreads) sample_draw_kernel(SampleArgs a)
{
    __shared__ DrawLds lds;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = blockIdx.x, req = row / a.T, t = row % a.T, V = a.V;
    const Settings set = load_settings(a, req);
    const int n_chunks = (V + kChunk - 1) / kChunk;
    const float u = a.uniforms[row];
    const bool drafted = a.accept && t < a.T - 1;
    const int d = drafted ? a.draft[(size_t)req * (a.T - 1) + t] : -1;
    const float xd = d >= 0 && d < V ? a.draft_logit[row] : kNegInf;

    const float *tops = a.tops + (size_t)row * n_chunks;
    float gm = kNegInf;
    for (int c = tid; c < n_chunks; c += kDrawThreads)
        gm = fmaxf(gm, tops[c]);
    gm = block_max(gm, lds.fl);
    Draw out = {-1, 0.0f, 0.0f};
    if (gm > kNegInf) {
        // the chunks' masses, the draft's apart
        const float *refs = a.refs + (size_t)row * n_chunks;
        const double *sums = a.sums + (size_t)row * n_chunks;
        float ref = kNegInf;
        u64 total = 0ull;
        auto chunk_mass = [&](int c) { return fixed(sums[c] * mass_below(refs[c], ref, set.inv_t), a.bits); };
        double whole = 0.0;                   // relative to gm, with the draft
        const double md = xd > kNegInf ? mass_below(xd, gm, set.inv_t) : 0.0;
        if (set.summed()) {
            for (int c = tid; c < n_chunks; c += kDrawThreads)
                ref = fmaxf(ref, refs[c]);
            ref = block_max(ref, lds.fl);
            u64 w = 0ull;
            if (ref > kNegInf)
                for (int c = tid; c < n_chunks; c += kDrawThreads)
                    w += chunk_mass(c);
            block_scan(w, lds.scan, total);
            whole = md + floating(total, a.bits) * (ref > kNegInf ? mass_below(ref, gm, set.inv_t) : 0.0);
        }
        if (!set.filtered()) {
            out.p_draft = (float)(md / whole);
            if (total) {
                const u64 target = drawn(u, total);
                u64 before = 0ull;
                for (int c0 = 0; c0 < n_chunks; c0 += kDrawThreads) {
                    const u64 w = c0 + tid < n_chunks ? chunk_mass(c0 + tid) : 0ull;
                    u64 part;
                    const u64 upto = before + block_scan(w, lds.scan, part);
                    if (upto - w <= target && target < upto) {
                        lds.at = c0 + tid;
                        lds.rest = target - (upto - w);
                        lds.found = w;
                    }
                    before += part;
                }
                __syncthreads();
                const int chunk = lds.at;
                const u64 rest = lds.rest, size = lds.found;
                // That chunk once more, under its rules: a token a thread.  In one far below
                // the best, tokens may have less than half a unit each, where their sum
                // has some: there masses are relative to the chunk's own largest, and the
                // target is the same part of their sum.
                const bool far = size < 1ull << 20;
                const float top = far ? refs[chunk] : ref;
                SliceWalk<kDtype> walk(a, lds.words, chunk * kChunk, kChunk, req, t, 0, 1);
                float *ruled = reinterpret_cast<float *>(lds.few);
                if (wave == 0) {
                    walk.load_request();
                    walk.rule(chunk * kChunk, walk.ha);
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        ruled[64 * i + lane] = walk.ha.x[i];
                }
                __syncthreads();
                const float x = drafted && chunk * kChunk + tid == d ? kNegInf : ruled[tid];
                const double mass = mass_below(x, top, set.inv_t);
                const u64 w = fixed_one(mass, a.bits);
                u64 all;
                const u64 upto = block_scan(w, lds.scan, all);
                // the chunk's sum may be up to 512 units off that of its tokens' units; the
                // row's last unit is its last token's
                u64 goal = target + 1ull == total ? all - 1ull : min(rest, all - 1ull);
                if (far && target + 1ull < total)
                    goal = min((u64)((double)rest * ((double)all / (double)size)), all - 1ull);
                if (upto - w <= goal && goal < upto) {
                    lds.at = chunk * kChunk + tid;
                    lds.value = (float)((far ? mass * mass_below(top, ref, set.inv_t) : mass) / floating(total, a.bits));
                }
                __syncthreads();
                out.token = lds.at;
                out.prob = lds.value;
            }
        } else {
            u64 *cand = a.cand + (size_t)row * V;
            const int n_cand = a.counts[row * kPad];
            const Row r = {a, set, gm, whole, d, u};
            if (n_cand <= kFew) {
                if (tid < n_cand)
                    lds.few[tid] = cand[tid];
                out = draw_few(r, n_cand, lds);
            } else if (!draw_binned(r, cand, n_cand, a.lows[row], lds, out)) {
                out = draw_many(r, [&](auto &&f) { each_of(cand, n_cand, f); }, lds);
            }
        }
    }
    if (tid == 0) {
        a.token_ids[row] = out.token;
        a.token_probs[row] = out.prob;
        if (a.accept) {
            if (drafted) {
                const size_t di = (size_t)req * (a.T - 1) + t;
                a.p_draft[di] = out.p_draft;
                __hip_atomic_store(&a.oks[row], a.accept[di] < out.p_draft ? 1u : 0u, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            }
            // the request's last row counts
            const uint32_t done = __hip_atomic_fetch_add(&a.tickets[req], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
            if (done == (uint32_t)a.T - 1u) {
                int k = 0;
                while (k < a.T - 1 && __hip_atomic_load(&a.oks[(size_t)req * a.T + k], __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT))
                    ++k;
                a.n_accepted[req] = k;
            }
        }
    }
}

// ---------------------------------------------------------------- host side

struct Layout {
    size_t cand, tops, bars, refs, sums, counts, lows, draft_logit, tickets, oks, bytes;
};

Layout layout_for(int R, int T, int V)
{
    Layout l;
    const size_t M = (size_t)R * T, chunks = (V + kChunk - 1) / kChunk;
    l.cand = 0;
    l.tops = round256(M * V * 8);
    l.bars = l.tops + round256(M * chunks * 4);
    l.refs = l.bars + round256(M * chunks * 4);
    l.sums = l.refs + round256(M * chunks * 4);
    l.counts = l.sums + round256(M * chunks * 8);
    l.lows = l.counts + round256(M * 4 * kPad);
    l.draft_logit = l.lows + round256(M * 4);
    l.tickets = l.draft_logit + round256(M * 4);
    l.oks = l.tickets + round256((size_t)R * 4);
    l.bytes = l.oks + round256(M * 4);
    return l;
}

// Whether a request may have a filter, as far as the host can tell.
bool may_filter(const int4vh_sampling &s)
{
    return s.temperatures || s.top_ks || s.top_ps || s.min_ps || !(s.temperature > 0.0f) || s.top_k > 0 ||
           s.top_p < 1.0f || s.min_p > 0.0f;
}

template <int kDtype>
hipError_t launch(const SampleArgs &a, const Shape &sh, hipStream_t s)
{
    hipLaunchKernelGGL(sample_scan_kernel<kDtype>, sh.grid, sh.block, sh.lds, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (may_filter(a.s)) {
        hipLaunchKernelGGL(sample_collect_kernel<kDtype>, sh.grid, sh.block, sh.lds, s, a);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(sample_draw_kernel<kDtype>, dim3(a.R * a.T), dim3(kDrawThreads), 0, s, a);
    return hipGetLastError();
}

} // namespace

extern "C" {

size_t sample_logits_workspace_bytes(int R, int T, int V)
{
    if (!sizes_ok(R, T, V) || V > kMaxV)
        return 0;
    return layout_for(R, T, V).bytes;
}

int sample_logits_rows(const void *logits, int64_t logits_stride, int dtype, const int32_t *draft_ids, int R, int T,
                       int V, const int4vh_logit_rules *rules, const int4vh_sampling *sampling, const float *uniforms,
                       const float *accept, int32_t *token_ids, float *token_probs, float *p_draft,
                       int32_t *n_accepted, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = check_rules(logits, logits_stride, dtype, draft_ids, R, T, V, rules);
    if (st == INT4VH_EINVAL)
        return st;
    if (!sampling || !uniforms || !token_ids || !token_probs || !workspace)
        return INT4VH_EINVAL;
    if (accept && (T == 1 || !p_draft || !n_accepted))
        return INT4VH_EINVAL;
    if (!sampling->temperatures && (!(sampling->temperature >= 0.0f) || !std::isfinite(sampling->temperature)))
        return INT4VH_EINVAL;
    if ((!sampling->top_ks && sampling->top_k < 0) ||
        (!sampling->top_ps && !(sampling->top_p >= 0.0f && sampling->top_p <= 1.0f)) ||
        (!sampling->min_ps && !(sampling->min_p >= 0.0f && sampling->min_p <= 1.0f)))
        return INT4VH_EINVAL;
    if (!rows_aligned(sampling->temperatures, 4) || !rows_aligned(sampling->top_ks, 4) ||
        !rows_aligned(sampling->top_ps, 4) || !rows_aligned(sampling->min_ps, 4) || !rows_aligned(uniforms, 4) ||
        !rows_aligned(accept, 4) || !rows_aligned(token_ids, 4) || !rows_aligned(token_probs, 4) ||
        !rows_aligned(p_draft, 4) || !rows_aligned(n_accepted, 4) || !rows_aligned(workspace, 256))
        return INT4VH_EALIGN;
    if (st != INT4VH_OK)
        return st;
    const Layout l = layout_for(R, T, V);
    if (workspace_bytes < l.bytes)
        return INT4VH_EWORKSPACE;
    int cus = 0;
    if ((st = current_cus(&cus)) != INT4VH_OK)
        return st;

    char *ws = static_cast<char *>(workspace);
    SampleArgs a = {};
    a.logits = logits;
    a.logits_stride = logits_stride;
    a.draft = draft_ids;
    a.R = R;
    a.T = T;
    a.V = V;
    fill_rules(a, rules, T);
    a.s = *sampling;
    a.uniforms = uniforms;
    a.accept = accept;
    int v_bits = 0;
    while ((1 << v_bits) < V)
        ++v_bits;
    a.bits = v_bits < 12 ? 50 : 62 - v_bits;
    a.cand = reinterpret_cast<u64 *>(ws + l.cand);
    a.tops = reinterpret_cast<float *>(ws + l.tops);
    a.bars = reinterpret_cast<float *>(ws + l.bars);
    a.refs = reinterpret_cast<float *>(ws + l.refs);
    a.sums = reinterpret_cast<double *>(ws + l.sums);
    a.counts = reinterpret_cast<int *>(ws + l.counts);
    a.lows = reinterpret_cast<float *>(ws + l.lows);
    a.draft_logit = reinterpret_cast<float *>(ws + l.draft_logit);
    a.tickets = reinterpret_cast<uint32_t *>(ws + l.tickets);
    a.oks = reinterpret_cast<uint32_t *>(ws + l.oks);
    a.token_ids = token_ids;
    a.token_probs = token_probs;
    a.p_draft = p_draft;
    a.n_accepted = n_accepted;
    const Shape sh = shape_for(a, 0, cus);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == INT4VH_ROWS_F32   ? launch<INT4VH_ROWS_F32>(a, sh, s)
                         : dtype == INT4VH_ROWS_F16 ? launch<INT4VH_ROWS_F16>(a, sh, s)
                                                    : launch<INT4VH_ROWS_BF16>(a, sh, s);
    return e == hipSuccess ? INT4VH_OK : hip_fail(e, "sampling kernel launch");
}

} // extern "C"
