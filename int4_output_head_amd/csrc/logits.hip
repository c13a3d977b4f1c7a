// logits.hip -- rules on logits (penalties for repeated tokens, biases,
// grammar masks) and verification under them, for MI355X (gfx950); formulas
// and order of rounding in int4vh_logits.h.
//
// Bound by HBM: the logits are read once (and written once by the apply
// call); a row of 151936 binary32 logits is 608 KB against a few KB of rules.
// The rules' cost is finding each token's count, which depends on the request
// and hardly on the row: a workgroup takes a slice of the vocabulary and
// several rows of ONE request and counts the slice's tokens of the request's
// history in LDS (integer atomics: any order gives the same counts).  Its
// waves then walk the slice, one or more to a row, 1024 tokens at a time with
// the next ones' loads in flight; a lane's tokens lie 64 apart, so that a
// mask's 64 bits are one scalar and a group without counts costs one test.
// The history is read once per slice and row group, from L2.
//
// Verification keeps one pass over the logits: each wave keeps its tokens'
// best keys in a small buffer, their (max, sum) and the draft's logit, and
// rules_merge_kernel joins the waves' lists of each row and counts accepted
// drafts.  The top-k goes by thresholds: at first the k-th largest of the 64
// lanes' maxima, which is at most the k-th value, then the k-th key held; the
// few values that reach it are ranked by counting the larger ones.  Exact for
// any input, ties included (keys are distinct, and a later token loses a tie).
//
// Measured (graph-timed, 64 requests x 4 rows of 151936 binary32 logits): the
// rules written out in 70 us (4.4 TB/s; a large copy reaches 4.7), without any
// rule in 67; verified greedily in 44.5 us and with top-16 in 61.5, without
// rules in 31 and 47.5 us (5.0 and 3.3 TB/s).  Of the 61.5 the penalties are 7,
// the mask 2, the bias 1, the merge 5.4; vector instructions take 62 % of the busy
// cycles.  One request's 16 rows, top-16, with a history of 25000 tokens take
// 25 us (with 1000: 20), the merge 7.7 of them.
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>

#include "int4vh.h"
#include "int4vh_internal.h"
#include "int4vh_logits.h"
#include "logits_common.h"
#include "rows_common.h"

#pragma clang fp contract(off)

namespace {

using namespace int4vh_detail;

constexpr int kMaxTopK = 16;
constexpr int kBuf = 128;                 // candidate keys per wave

struct RowsArgs : RulesArgs {
    // apply
    void *out;
    long long out_stride;
    // verify
    int top_k;
    float lse_scale;           // log2(e) / temperature
    u64 *lists;                // [R*T, n_lists, max(top_k, 1)] best keys of each wave's tokens, best first, 0 past the last
    u64 *heads;                // [R*T, n_lists] the lists' first keys (top_k >= 1)
    float2 *sums;              // [R*T, n_lists] (max, sum of exp2((x - max) * lse_scale))
    float *draft_logit;        // [R*T] ruled logit of the row's draft, where it is in [0, V)
};

// Keeps the k best of the n (<= kBuf) distinct keys buf[0, n), best first, and
// returns how many there are (min(n, k)).  A key's rank is the number of
// larger ones, which pass by in scalar registers.  Called by a whole wave on
// its own buffer.
__device__ __forceinline__ int keep_best(u64 *buf, int n, int k, int lane)
{
    const u64 a = lane < n ? buf[lane] : 0ull;
    int ra = 0;
    // four at a time: lanes past n hold key 0, which is larger than none
    if (n <= 64) {
#pragma nounroll
        for (int i = 0; i < n; i += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ra += readlane64(a, i + j) > a;
    } else {
        const u64 b = lane + 64 < n ? buf[lane + 64] : 0ull;
        int rb = 0;
#pragma nounroll
        for (int i = 0; i < 64; i += 2)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u64 o = readlane64(a, i + j), q = readlane64(b, i + j);
                ra += (o > a) + (q > a);
                rb += (o > b) + (q > b);
            }
        if (lane + 64 < n && rb < k)
            buf[rb] = b;
    }
    // (a lane's own keys are in registers: no read follows these writes)
    if (lane < n && ra < k)
        buf[ra] = a;
    wave_fence();
    return n < k ? n : k;
}

// Appends the keys of the lanes in `mask`; a buffer that could overflow is
// first cut to its k best.  Wave-uniform control flow.
__device__ __forceinline__ void push(u64 *buf, int &n, u64 key, u64 mask, int k, int lane)
{
    if (n + __popcll(mask) > kBuf) {
        n = keep_best(buf, n, k, lane);
        if (n == k) {
            const u64 last = buf[k - 1];
            mask &= __ballot(key > last);
        }
    }
    if (mask >> lane & 1ull)
        buf[n + lane_rank(mask)] = key;
    wave_fence();
    n += __popcll(mask);
}

// Appends those of every lane's kN keys whose value reaches the word th (above
// 0): a lane's place is the sum of the lower lanes' numbers, taken bit by bit.
template <int kN>
__device__ __forceinline__ void push_some(u64 *buf, int &n, const u64 (&key)[kN], uint32_t th, int k,
                                          int lane)
{
    uint32_t mine = 0u;
#pragma unroll
    for (int u = 0; u < kN; ++u)
        mine += (uint32_t)(key[u] >> 32) >= th ? 1u : 0u;
    int at = n, all = n;
#pragma unroll
    for (int b = 0; (1 << b) <= kN; ++b) {
        const u64 m = __ballot((mine >> b & 1u) != 0u);
        at += lane_rank(m) << b;
        all += __popcll(m) << b;
    }
    if (all <= kBuf) {
#pragma unroll
        for (int u = 0; u < kN; ++u)
            if ((uint32_t)(key[u] >> 32) >= th)
                buf[at++] = key[u];
        n = all;
        wave_fence();
    } else {
        // one at a time, in one copy of the code: the keys move down
        u64 rest[kN];
#pragma unroll
        for (int u = 0; u < kN; ++u)
            rest[u] = key[u];
#pragma nounroll
        for (int i = 0; i < kN; ++i) {
            push(buf, n, rest[0], __ballot((uint32_t)(rest[0] >> 32) >= th), k, lane);
#pragma unroll
            for (int u = 0; u + 1 < kN; ++u)
                rest[u] = rest[u + 1];
        }
    }
}

// The rows under the rules (SliceWalk).  kVerify: reduce the rows; otherwise
// write them out.
template <int kDtype, bool kVerify, bool kTopK, bool kLse>
__global__ void __launch_bounds__(64 * kMaxWaves) rules_kernel(RowsArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint32_t s_mem[];
    SliceWalk<kDtype> walk(a, s_mem);
    if (!walk.live())
        return;                               // no barrier follows
    walk.load_request();
    const int lane = walk.lane, row = walk.row, way = walk.way, d = walk.d, V = a.V;
    constexpr size_t kSize = SliceWalk<kDtype>::kSize;
    u64 *buf = reinterpret_cast<u64 *>(walk.entries + (a.has_penalty || a.has_bias ? a.slice : 0)) +
               __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kBuf;

    int n = 0;                                // keys in buf
    float above = kNegInf;                    // once k keys are held: a value has to be at least this
    float bv = kNegInf;                       // this lane's largest value, and its lowest token
    int bt = -1;
    float lm = kNegInf, ls = 0.0f;            // this lane's (max, sum)

    walk.run([&](int chunk0, float (&x)[kPer]) {
        if constexpr (!kVerify) {
            char *orow = static_cast<char *>(a.out) + (size_t)row * a.out_stride * kSize;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (chunk0 + 64 * i + lane < V)
                    store_logit<kDtype>(orow, chunk0 + 64 * i + lane, x[i]);
            return;
        }
        float best = kNegInf;                 // fmaxf passes over NaN
        if constexpr (kTopK || kLse) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                best = fmaxf(best, x[i]);
        }
        if constexpr (kLse) {
            const float m = fmaxf(lm, best);
            ls *= exp2_below(lm, m, a.lse_scale);
            lm = m;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                ls += exp2_below(x[i], m, a.lse_scale);
            ls = m > kNegInf ? ls : 0.0f;
        }
        if constexpr (kTopK) {
            // the values from `from` on are candidates: before k keys are held,
            // those that reach the chunk's threshold
            const int k = a.top_k;
            float from = above;
            if (n < k) {
                const uint32_t th = reach_threshold(best > kNegInf ? order_word(best) : 0u, k);
                from = th > 1u ? word_value(th) : -3.402823466e38f;
            }
            if (__ballot(best >= from)) {
                u64 m[kPer];
                int count = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    m[i] = __ballot(x[i] >= from);
                    count += __popcll(m[i]);
                }
                if (n + count <= kBuf) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (m[i]) {
                            if (x[i] >= from)
                                buf[n + lane_rank(m[i])] = order_key(x[i], chunk0 + 64 * i + lane);
                            n += __popcll(m[i]);
                        }
                    wave_fence();
                } else {
                    // one at a time, in one copy of the code: the values move down
                    float rest[kPer];
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        rest[i] = x[i];
#pragma nounroll
                    for (int i = 0; i < kPer; ++i) {
                        push(buf, n, order_key(rest[0], chunk0 + 64 * i + lane), __ballot(rest[0] >= from), k, lane);
#pragma unroll
                        for (int j = 0; j + 1 < kPer; ++j)
                            rest[j] = rest[j + 1];
                    }
                }
                if (above == kNegInf || n > 48) {
                    n = keep_best(buf, n, k, lane);
                    // later tokens lose a tie: the next larger value
                    if (n == k)
                        above = word_value((uint32_t)(buf[k - 1] >> 32) + 1u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const bool more = x[i] > bv;
                bv = more ? x[i] : bv;
                bt = more ? chunk0 + 64 * i + lane : bt;
            }
        }
        const uint32_t da = (uint32_t)d - (uint32_t)chunk0;
        if (d >= 0 && d < V && da < (uint32_t)kChunk) {
            float v = kNegInf;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                v = (int)(da >> 6) == i ? x[i] : v;
            if ((int)(da & 63u) == lane)
                a.draft_logit[row] = v;
        }
    });

    if constexpr (kVerify) {
        const size_t slot = (size_t)row * a.n_lists + blockIdx.x * a.ways + way;
        if constexpr (kLse) {
            const float m = wave_max(lm);
            const float s = wave_sum(ls * exp2_below(lm, m, a.lse_scale));
            if (lane == 0)
                a.sums[slot] = make_float2(m, m > kNegInf ? s : 0.0f);
        }
        if constexpr (kTopK) {
            const int k = a.top_k;
            if (n > k)
                n = keep_best(buf, n, k, lane);
            const u64 key = lane < n ? buf[lane] : 0ull;
            if (lane < k)
                a.lists[slot * k + lane] = key;
            if (lane == 0)
                a.heads[slot] = key;
        } else {
            const u64 key = wave_max64(bt >= 0 ? order_key(bv, bt) : 0ull);
            if (lane == 0)
                a.lists[slot] = key;
        }
    }
}

struct MergeArgs {
    const u64 *lists, *heads;
    const float2 *sums;
    const float *draft_logit;
    const int32_t *draft;
    const float *draft_probs, *uniforms;   // both or neither
    int R, T, V, top_k, n_lists;
    float temperature, lse_scale;
    float *logits_max;
    int32_t *argmax, *topk_ids;
    float *topk_logits, *lse, *p_draft;
    int32_t *n_acc;
};

// One workgroup per request, one wave per row: the row's lists joined, then
// the request's accepted count.  A few hundred or thousand keys a row, from
// other XCDs' caches: latency counts.  Up to 64 lists are loaded at once, 16
// lanes a list, and their first keys meet in LDS for the threshold.  Of more
// lists (a short call's rows are cut into many) the first keys alone come
// first, and then the lists that reach the threshold: one compute unit would
// take longer for all of them (149 lists of 16 rows: 14.4 us, so 7.7).
constexpr int kHeads = 4;                     // first keys per lane at a time

// kMany: a top-k call of more than 64 lists a row.
template <bool kTopK, bool kLse, bool kMany>
__global__ void __launch_bounds__(64 * 16) rules_merge_kernel(MergeArgs a)
{
    __shared__ u64 s_buf[kTopK ? 16 : 1][kBuf];
    __shared__ uint32_t s_head[kTopK && !kMany ? 16 : 1][64];
    __shared__ int s_open[kMany ? 16 : 1][64 * kHeads];
    __shared__ int s_ok[16];
    const int lane = threadIdx.x & 63, t = threadIdx.x >> 6, req = blockIdx.x;
    const int row = req * a.T + t;
    const int n_lists = a.n_lists;
    const bool drafted = t < a.T - 1;
    const size_t di = drafted ? (size_t)req * (a.T - 1) + t : 0;
    const int d = drafted ? a.draft[di] : -1;
    const float bar = drafted && a.draft_probs ? a.uniforms[di] * a.draft_probs[di] : 0.0f;

    const int k = kTopK ? a.top_k : 1;
    const u64 *lists = a.lists + (size_t)row * n_lists * k;
    constexpr int kKeys = kTopK ? kMaxTopK : 1;
    u64 key[kKeys];                           // of the (i0 + 4u + lane / 16)-th of n lists; greedy: the lane-th
    auto load_lists = [&](int i0, int n, const int *open) {
        const int rank = kTopK ? lane & 15 : 0, first = kTopK ? lane >> 4 : lane;
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int i = min(i0 + 4 * u + first, n - 1);
            key[u] = lists[(uint32_t)((open ? open[i] : i) * k + min(rank, k - 1))];
        }
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
            key[u] = i0 + 4 * u + first < n && rank < k ? key[u] : 0ull;
    };
    if constexpr (!kMany)
        load_lists(0, n_lists, nullptr);
    float gm = kNegInf, gs = 0.0f;
    if constexpr (kLse) {
        const float2 *sums = a.sums + (size_t)row * n_lists;
        for (int c = lane; c < n_lists; c += 64)
            gm = fmaxf(gm, sums[c].x);
        gm = wave_max(gm);
        for (int c = lane; c < n_lists; c += 64) {
            const float2 p = sums[c];
            gs += p.y * exp2_below(p.x, gm, a.lse_scale);
        }
        gs = wave_sum(gs);
        if (a.lse && lane == 0)
            a.lse[row] = gs > 0.0f ? gm / a.temperature + logf(gs) : kNegInf;
    }

    float p = 0.0f;
    u64 top;                                  // the row's best key
    if constexpr (kTopK) {
        u64 *buf = s_buf[t];
        int n = 0;
        if constexpr (!kMany) {
            if ((lane & 15) == 0)
#pragma unroll
                for (int u = 0; u < kKeys; ++u)
                    s_head[t][4 * u + (lane >> 4)] = (uint32_t)(key[u] >> 32);
            wave_fence();
            push_some(buf, n, key, reach_threshold(s_head[t][lane], k), k, lane);
        } else {
            int *open = s_open[t];
            const u64 *heads = a.heads + (size_t)row * n_lists;
            u64 h[kHeads], best = 0ull;
            auto load_heads = [&](int c0) {
#pragma unroll
                for (int u = 0; u < kHeads; ++u)
                    h[u] = heads[min(c0 + 64 * u + lane, n_lists - 1)];
#pragma unroll
                for (int u = 0; u < kHeads; ++u)
                    h[u] = c0 + 64 * u + lane < n_lists ? h[u] : 0ull;
            };
            for (int c0 = 0; c0 < n_lists; c0 += 64 * kHeads) {
                load_heads(c0);
#pragma unroll
                for (int u = 0; u < kHeads; ++u)
                    best = h[u] > best ? h[u] : best;
            }
            const uint32_t th = reach_threshold((uint32_t)(best >> 32), k);
            for (int c0 = 0; c0 < n_lists; c0 += 64 * kHeads) {
                if (n_lists > 64 * kHeads)
                    load_heads(c0);
                int n_open = 0;
#pragma unroll
                for (int u = 0; u < kHeads; ++u) {
                    const bool reach = (uint32_t)(h[u] >> 32) >= th;
                    const u64 m = __ballot(reach);
                    if (reach)
                        open[n_open + lane_rank(m)] = c0 + 64 * u + lane;
                    n_open += __popcll(m);
                }
                wave_fence();
                for (int i0 = 0; i0 < n_open; i0 += 64) {
                    load_lists(i0, n_open, open);
                    push_some(buf, n, key, th, k, lane);
                }
                wave_fence();
            }
        }
        n = keep_best(buf, n, k, lane);
        const u64 mine = lane < n ? buf[lane] : 0ull;
        top = readlane64(mine, 0);
        const float v = mine ? key_value(mine) : kNegInf;
        const int id = mine ? key_token(mine) : -1;
        if (lane < k) {
            a.topk_ids[(size_t)row * k + lane] = id;
            a.topk_logits[(size_t)row * k + lane] = v;
        }
        if (a.draft_probs && drafted) {
            float e = mine ? exp2_below(v, key_value(top), a.lse_scale) : 0.0f, e_d = id == d ? e : 0.0f;
#pragma unroll
            for (int off = 8; off >= 1; off >>= 1) {          // the keys are in the first 16 lanes
                e += __shfl_xor(e, off);
                e_d += __shfl_xor(e_d, off);
            }
            p = n ? e_d / e : 0.0f;
        }
    } else {
        u64 best = key[0];
        for (int c = 64 + lane; c < n_lists; c += 64)
            best = lists[c] > best ? lists[c] : best;
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
                ok = bar < p;
            } else {
                ok = id >= 0 && id == d;
            }
        }
        s_ok[t] = ok;
    }
    __syncthreads();
    if (t == 0) {
        const u64 accepted = __ballot(lane < a.T - 1 && s_ok[lane < 16 ? lane : 0]);
        if (lane == 0)
            a.n_acc[req] = __builtin_ctzll(~accepted);        // the leading ones
    }
}

// ---------------------------------------------------------------- host side

struct Layout {
    size_t lists, heads, sums, draft_logit, bytes;
};

Layout layout_for(int R, int T, int V, int top_k)
{
    Layout l;
    // a list covers kChunk tokens at least, but for those past the vocabulary's
    // end in the last slice
    const size_t M = (size_t)R * T, n = (V + kChunk - 1) / kChunk + kMaxWaves;
    l.lists = 0;
    l.heads = round256(M * n * 8 * (top_k ? top_k : 1));
    l.sums = l.heads + (top_k ? round256(M * n * 8) : 0);
    l.draft_logit = l.sums + round256(M * n * 8);
    l.bytes = l.draft_logit + round256(M * 4);
    return l;
}

template <bool kVerify, bool kTopK, bool kLse>
hipError_t launch_rules(const RowsArgs &a, int dtype, const Shape &sh, hipStream_t s)
{
    void (*k)(RowsArgs) = dtype == INT4VH_ROWS_F32   ? rules_kernel<INT4VH_ROWS_F32, kVerify, kTopK, kLse>
                           : dtype == INT4VH_ROWS_F16 ? rules_kernel<INT4VH_ROWS_F16, kVerify, kTopK, kLse>
                                                      : rules_kernel<INT4VH_ROWS_BF16, kVerify, kTopK, kLse>;
    hipLaunchKernelGGL(k, sh.grid, sh.block, sh.lds, s, a);
    return hipGetLastError();
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
    int st = check_rules(logits, logits_stride, dtype, draft_ids, R, T, V, rules);
    if (st != INT4VH_OK)
        return st;
    if (!rows_aligned(out, rows_size(dtype)))
        return INT4VH_EALIGN;
    int cus = 0;
    if ((st = current_cus(&cus)) != INT4VH_OK)
        return st;
    RowsArgs a = {};
    a.logits = logits;
    a.logits_stride = logits_stride;
    a.draft = draft_ids;
    a.R = R;
    a.T = T;
    a.V = V;
    a.out = out;
    a.out_stride = out_stride;
    fill_rules(a, rules, T);
    const Shape sh = shape_for(a, 0, cus);
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
    int st = check_rules(logits, logits_stride, dtype, draft_ids, R, T, V, rules);
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
    RowsArgs a = {};
    a.logits = logits;
    a.logits_stride = logits_stride;
    a.draft = draft_ids;
    a.R = R;
    a.T = T;
    a.V = V;
    fill_rules(a, rules, T);
    a.top_k = top_k;
    a.lse_scale = 1.4426950408889634f / temperature;
    a.lists = reinterpret_cast<u64 *>(ws + l.lists);
    a.heads = reinterpret_cast<u64 *>(ws + l.heads);
    a.sums = reinterpret_cast<float2 *>(ws + l.sums);
    a.draft_logit = reinterpret_cast<float *>(ws + l.draft_logit);
    const Shape sh = shape_for(a, top_k > 0 ? kBuf * 8 : 0, cus);
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
    m.lists = a.lists;
    m.heads = a.heads;
    m.sums = a.sums;
    m.draft_logit = a.draft_logit;
    m.draft = draft_ids;
    m.draft_probs = sampled ? draft_probs : nullptr;
    m.uniforms = sampled ? uniforms : nullptr;
    m.R = R;
    m.T = T;
    m.V = V;
    m.top_k = top_k;
    m.n_lists = a.n_lists;
    m.temperature = temperature;
    m.lse_scale = a.lse_scale;
    m.logits_max = logits_max;
    m.argmax = argmax_ids;
    m.topk_ids = topk_ids;
    m.topk_logits = topk_logits;
    m.lse = lse;
    m.p_draft = p_draft;
    m.n_acc = n_accepted;
    const bool many = a.n_lists > 64;
    void (*k)(MergeArgs) = !top_k ? (want_lse ? rules_merge_kernel<false, true, false> : rules_merge_kernel<false, false, false>)
                           : many ? (want_lse ? rules_merge_kernel<true, true, true> : rules_merge_kernel<true, false, true>)
                                  : (want_lse ? rules_merge_kernel<true, true, false> : rules_merge_kernel<true, false, false>);
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
    int st = check_rules(ws, V, INT4VH_ROWS_F32, draft_ids, R, T, V, rules);
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
