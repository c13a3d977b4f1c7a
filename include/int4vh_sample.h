/*
 * int4vh_sample.h -- C ABI of the sampler: a token of every row drawn by a given
 * uniform number at a temperature, among the top k, the top p and those above
 * min p, under the rules of int4vh_logits.h, and drafted tokens verified with
 * the same distribution (same library, libint4vh.so; status codes and error
 * text as in int4vh.h).
 *
 * Rows, drafts and rules are those of int4vh_logits.h.  For each row, with x the
 * ruled logits, NaN counted as -infinity, and the settings of its request:
 *
 *   best     = the largest x, of equal ones the lowest token
 *   mass(v)  = exp((x[v] - x[best]) / temperature); 1 where x[v] = x[best]
 *   1. top_k: the top_k tokens of largest x (ties: the lower token)
 *   2. top_p: of these, from the best on, those whose predecessors' mass is below
 *      top_p times the mass of all of step 1; the best always
 *   3. min_p: of these, those with mass >= min_p
 *
 *   token    = the first, by token id, at which the sum of the kept tokens' mass
 *              exceeds uniforms[row] times their whole mass
 *   prob     = its mass, divided by that whole
 *
 * A temperature that is 0 (or, from a device array, negative or not finite) keeps the
 * best token alone; a top_k of 0 or less, a top_p of 1 or more and a min_p of 0
 * or less keep all; a min_p above 1 counts as 1.  A uniform number below 0 counts
 * as 0, one of 1 or more as the largest below 1.  A row with nothing above
 * -infinity has token -1 and prob 0.  Tokens of +infinity share the row alike.
 *
 * Drafts.  With accept (uniform numbers of the drafts, [R, T-1]) the drafts are
 * verified as point masses, those of a copy from the context or of a greedy
 * drafter:
 *   p_draft [R, T-1]   d's mass, if it is kept, divided by the whole; 0 otherwise
 *   n_accepted [R]     leading drafts with accept < p_draft
 *   and in rows with a draft the token is another one: d's mass counts as 0 there
 *   (-1 and prob 0 where nothing else is left), so that token_ids[n_accepted] of a
 *   request is the token behind its accepted drafts.
 * Without it, every row's token comes from all that is kept.
 *
 * Numerics.  The ruled logits are binary32; masses are computed in binary64, to
 * 2^-40 of each, and added as whole multiples of 2^-b, b = 62 - ceil(log2(V)) (44
 * for 151936 tokens) and at most 50, so that sums do not depend on an order.  Under
 * top_k, top_p or min_p a kept token's mass below half of that counts as none, and
 * the token is not drawn.  Without them, and for the mass of a whole row that top_p
 * is a part of, sums of 1024 tokens (binary64, in a fixed order) are rounded to
 * multiples of 2^-b, and a token is found among its 1024 by masses in these units, or,
 * where the sum has less than 2^20 of them, relative to the largest of the 1024: those
 * far below the best keep their share.  Results are the same in every run.
 *
 * Calls are asynchronous on `stream`, allocate nothing and may be captured in a
 * graph.  Errors: as in int4vh_logits.h, and INT4VH_EINVAL for NULL uniforms,
 * token_ids, token_probs or sampling, accept without drafts (T == 1) or without
 * p_draft and n_accepted, and a scalar setting that is out of range (temperature
 * negative or not finite, top_k negative, top_p or min_p outside [0, 1]).
 */
#ifndef INT4VH_SAMPLE_H
#define INT4VH_SAMPLE_H

#include <stddef.h>
#include <stdint.h>

#include "int4vh_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The requests' settings: device arrays of R values, or, where one is NULL, a
 * value for all of them.  The struct itself is host memory, read during the call. */
typedef struct int4vh_sampling {
    const float *temperatures;
    const int32_t *top_ks;
    const float *top_ps;
    const float *min_ps;
    float temperature;
    int32_t top_k;
    float top_p;
    float min_p;
} int4vh_sampling;

/* Bytes of workspace sample_logits_rows needs (0 if the sizes are invalid): 8 for
 * each logit, whatever the settings, and little else.  Pure host function.
 * 256-byte aligned, no initialisation; its contents mean nothing between calls.
 * Calls in flight at the same time must not share it. */
size_t sample_logits_workspace_bytes(int R, int T, int V);

int sample_logits_rows(const void *logits, int64_t logits_stride, int dtype, const int32_t *draft_ids, int R, int T,
                       int V, const int4vh_logit_rules *rules, const int4vh_sampling *sampling, const float *uniforms,
                       const float *accept, int32_t *token_ids, float *token_probs, float *p_draft,
                       int32_t *n_accepted, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* INT4VH_SAMPLE_H */
