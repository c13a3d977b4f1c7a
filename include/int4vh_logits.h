/*
 * int4vh_logits.h -- C ABI of the rules on logits behind the output head:
 * penalties for repeated tokens, biases and grammar masks, and verification
 * under them (same library, libint4vh.so; status codes and error text as in
 * int4vh.h).
 *
 * Rows are the positions of verify blocks, as in int4vh.h: request i owns rows
 * i*T .. i*T+T-1, and draft_ids [R, T-1] are its drafted tokens.  Row t of a
 * request is the position behind its drafts 0 .. t-1, so those count as
 * generated there.  For token v of row (i, t):
 *
 *   count  = occurrences of v among the request's generated tokens (its history
 *            from n_prompt[i] on) and its drafts 0 .. t-1
 *   seen   = v occurs there or anywhere in the request's history
 *   l0     = f32(logit)
 *   l1     = seen ? (l0 > 0 ? l0 / repetition[i] : l0 * repetition[i]) : l0
 *   l2     = count > 0 ? l1 - frequency[i] * count : l1
 *   l3     = count > 0 ? l2 - presence[i] : l2
 *   l4     = l3 + bias(i, v)
 *   ruled  = v is allowed in the row ? l4 : -infinity
 *
 * binary32, one rounding per operation in the order written (no fused
 * multiply-adds).  The mask selects: whatever a refused token's logit is, NaN
 * and infinities among it, its ruled value is -infinity.
 *
 * int4vh_logit_rules (device pointers; the struct itself is host memory, read
 * during the call):
 *   history          int32 [n_history], the requests' tokens back to back (prompt,
 *                    then generated), request i's in history[history_offsets[i]
 *                    .. history_offsets[i+1]); offsets int64 [R+1], clamped to
 *                    [0, n_history].  Ids outside [0, V) are ignored, here and
 *                    in draft_ids.  NULL: no history (drafts still count).
 *   n_prompt         int32 [R], leading tokens of each history that are the
 *                    prompt; NULL: 0, all of it is generated
 *   repetition, frequency, presence
 *                    float32 [R], each NULL for none; repetition > 0; infinite
 *                    ones hold too (a frequency or presence of infinity bans
 *                    what was generated, and nothing else)
 *   bias_ids, bias_values
 *                    int32, float32 [n_bias], request i's entries in
 *                    [bias_offsets[i], bias_offsets[i+1]) (int64 [R+1], clamped);
 *                    of entries with the same id the last one holds; ids outside
 *                    [0, V) are ignored.  NULL: none
 *   mask             uint32 [n_masks, mask_stride]: bit v % 32 of word v / 32 is 1
 *                    where token v is allowed.  NULL: every token is
 *   mask_index       int32 [R*T]: the mask of each row; negative: the row is
 *                    free; n_masks or more: nothing is allowed.  NULL: row r's
 *                    mask is mask r (n_masks >= R*T)
 *
 * Calls are asynchronous on `stream`, allocate nothing and may be captured in
 * a graph.
 *
 * Errors (host validation before any launch): INT4VH_EINVAL for T outside
 * [1, 16], R < 1, R*T > 4096, V < 1, an unknown dtype, a stride below V (R*T >
 * 1), a required pointer that is NULL (draft_ids when T > 1; the offsets with
 * a history or biases; a mask's words below ceil(V/32) or n_masks < 1, or below
 * R*T without mask_index; negative n_history or n_bias); INT4VH_EALIGN for a
 * pointer not aligned to its element; INT4VH_EUNSUPPORTED for V > 2^24,
 * n_history > 2^31 - 17 or n_bias > 2^31 - 1; INT4VH_EWORKSPACE, INT4VH_EHIP as
 * in int4vh.h.
 */
#ifndef INT4VH_LOGITS_H
#define INT4VH_LOGITS_H

#include <stddef.h>
#include <stdint.h>

#include "int4vh_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct int4vh_logit_rules {
    const int32_t *history;
    int64_t n_history;
    const int64_t *history_offsets;
    const int32_t *n_prompt;
    const float *repetition;
    const float *frequency;
    const float *presence;
    const int32_t *bias_ids;
    const float *bias_values;
    int64_t n_bias;
    const int64_t *bias_offsets;
    const uint32_t *mask;
    int64_t n_masks;
    int64_t mask_stride;
    const int32_t *mask_index;
} int4vh_logit_rules;

/* The ruled logits written out, for a sampler of the caller's own: logits
 * [R*T, V] and out [R*T, V] of `dtype` (INT4VH_ROWS_*), rows logits_stride /
 * out_stride elements apart; rounded once.  out may be logits itself with the
 * same stride, and may overlap nothing else.  rules NULL: none. */
int logit_rules_apply(const void *logits, int64_t logits_stride, int dtype, const int32_t *draft_ids, int R, int T,
                      int V, const int4vh_logit_rules *rules, void *out, int64_t out_stride, void *stream);

/* Bytes of workspace logit_rules_verify needs (0 if the sizes are invalid).
 * Pure host function.  256-byte aligned, no initialisation; its contents mean
 * nothing between calls.  Calls in flight at the same time must not share it. */
size_t logit_rules_verify_workspace_bytes(int R, int T, int V, int top_k);

/* Verification of the drafts under the rules, in one pass over the logits
 * (nothing is written back).  Outputs as verify_lm_head_int4_sampled, over the
 * ruled logits (ties: the lower token first):
 *   argmax_ids, logits_max  [R*T]; a row with nothing above -infinity has id -1
 *                           and -infinity
 *   topk_ids, topk_logits   [R*T, top_k], top_k in [0, min(16, V)]; ranks past the
 *                           row's tokens above -infinity hold -1 and -infinity
 *   lse                     [R*T] or NULL: log sum_v exp(ruled / temperature);
 *                           -infinity for an empty row
 * and with draft_probs and uniforms (float32 [R, T-1], both or neither):
 *   p_draft [R, T-1]        d's probability among the top_k (top_k >= 1) or the
 *                           whole vocabulary (top_k == 0); 0 for an id outside
 *                           [0, V) or a refused one
 *   n_accepted [R]          leading drafts with uniforms * draft_probs < p_draft
 * Without them the drafts are verified greedily, n_accepted[i] counting the
 * leading drafts that equal their row's argmax, and p_draft is not written
 * (NULL allowed).
 * A NaN in an allowed place is never chosen and counts as -infinity; rows
 * with +infinity split their probability among those tokens.
 * Errors as above, plus INT4VH_EINVAL for top_k out of range, a temperature
 * that is not finite and > 0, or one of draft_probs and uniforms alone. */
int logit_rules_verify(const void *logits, int64_t logits_stride, int dtype, const int32_t *draft_ids,
                       const float *draft_probs, const float *uniforms, int R, int T, int V,
                       const int4vh_logit_rules *rules, int top_k, float temperature, float *logits_max,
                       int32_t *argmax_ids, int32_t *topk_ids, float *topk_logits, float *lse, float *p_draft,
                       int32_t *n_accepted, void *workspace, size_t workspace_bytes, void *stream);

/* The head and the verification under rules in one call: the logits of
 * verify_lm_head_int4_batch (written to the workspace) go through
 * logit_rules_verify.  hidden, packed_w, scales as in int4vh.h.  The workspace
 * holds verify_lm_head_int4_ruled_workspace_bytes(R, T, V, H, top_k) bytes,
 * initialised once with verify_lm_head_int4_workspace_init. */
size_t verify_lm_head_int4_ruled_workspace_bytes(int R, int T, int V, int H, int top_k);

int verify_lm_head_int4_ruled(const void *hidden, const uint8_t *packed_w, const void *scales,
                              const int32_t *draft_ids, const float *draft_probs, const float *uniforms, int R, int T,
                              int V, int H, const int4vh_logit_rules *rules, int top_k, float temperature,
                              float *logits_max, int32_t *argmax_ids, int32_t *topk_ids, float *topk_logits,
                              float *lse, float *p_draft, int32_t *n_accepted, void *workspace,
                              size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* INT4VH_LOGITS_H */
