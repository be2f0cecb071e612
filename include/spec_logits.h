/*
 * spec_logits.h -- C ABI of what stands between the target model's logits and spec_verify: each
 * request's own rules about tokens.
 *
 * Sources (the same pages as spec_verify.h):
 *  - FreeToken PR #836, section "Design": every verify row follows its own request's sampling
 *    parameters, and penalties count the drafts before the row as already generated.
 *  - "Adding Speculative Decoding", "Verification and sampling": one batched call over k + 1 rows
 *    per request, requests with different k; the extra token honours the penalties.
 *
 * Conventions are those of spec_verify.h and spec_cache.h: device pointers, no allocation, no host
 * copy, no synchronisation, host-visible errors returned with nothing enqueued, device-data errors in
 * the workspace's sticky error word, no trap or assert.  The kernel is a programmatic dependent of the work
 * before it on its stream.  A call may be captured into a graph.
 */
#ifndef SPEC_LOGITS_H
#define SPEC_LOGITS_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device-data error codes of this call, beside SV_DEV_BAD_LAYOUT, _TOKEN, _PENALTY and _HISTORY. */
enum {
    SV_DEV_BAD_BIAS = 12,   /* bias offsets decrease or pass bias_len, or an id is outside [0, V) or
                               does not ascend                                                  */
    SV_DEV_BAD_MASK = 13    /* a row's mask index outside [-1, num_masks)                       */
};

/* The requests' rules: structure of device arrays, any group of them NULL for none. */
typedef struct sv_logit_rules {
    const float *repetition;        /* [B], > 0: divides positive logits of seen tokens, multiplies others */
    const float *presence;          /* [B]: subtracted once from a token that was generated     */
    const float *frequency;         /* [B]: subtracted per time that it was                      */
    /* Each request's history, as in sv_params, except that a count may be 0: the token was seen (in
     * the prompt), and only the repetition penalty looks at it. */
    const int32_t *prior_offsets;   /* [B + 1]                                                   */
    const int32_t *prior_tokens;    /* [prior_len] distinct ids per request, ascending           */
    const int32_t *prior_counts;    /* [prior_len] >= 0                                          */
    int32_t prior_len;
    int32_t bias_len;
    const int32_t *bias_offsets;    /* [B + 1], as prior_offsets                                 */
    const int32_t *bias_tokens;     /* [bias_len] distinct ids per request, ascending            */
    const float *bias_values;       /* [bias_len]                                                */
    /* Grammar masks, a bit per token: token v of mask m is allowed iff bit v % 32 of word
     * m * mask_words + v / 32 is set.  Bits from V on are not looked at. */
    const uint32_t *masks;          /* [num_masks, mask_words]                                   */
    const int32_t *mask_rows;       /* [total_rows]: the row's mask, or -1: every token allowed  */
    int32_t num_masks;
    int32_t mask_words;             /* >= (V + 31) / 32                                          */
} sv_logit_rules;

/*
 * spec_logits -- penalties for repeated tokens, biases and grammar masks on the logits of a verify
 * step, in one pass.
 *
 * For row i of request b and token v, with c = the token's count in the request's history plus its
 * count among the request's drafts before row i, and v "seen" iff it is one of those:
 *     z = logit
 *     z = z > 0 ? z / repetition : z * repetition        if v is seen
 *     z = z - (presence * [c > 0] + frequency * c)
 *     z = z + bias of v
 *     z = -inf                                           if the row's mask refuses v
 * Arithmetic is fp32, rounded once; a logit that no rule touches is copied bit by bit.  With
 * presence and frequency here, spec_verify is given none.  A row whose mask refuses everything is all
 * -inf, which spec_verify calls a row without a distribution.
 *
 *   logits       device [total_rows, V], dtype SV_BF16 or SV_F32, 16-byte aligned.
 *   draft_tokens device int32 [total_rows - B], num_drafts [B], row_offsets [B + 1] or NULL, B, k_max, V,
 *                total_rows: as in spec_verify.  draft_tokens may be NULL where no penalty is given.
 *   out          device, as logits, 16-byte aligned; may be logits itself: then only what changes is
 *                written.  Any other overlap is SV_ERR_INVALID_ARG.  Rows that no request uses are left as they were.
 *   workspace    its header only (256 bytes, 256-byte aligned); the call adds to its error word and
 *                does not clear it.
 * A request with a device-data error (SV_DEV_BAD_LAYOUT; SV_DEV_BAD_TOKEN: a draft outside [0, V), where
 * penalties are given; SV_DEV_BAD_PENALTY: one that is not finite, or repetition <= 0; offsets of its
 * history or bias out of range; SV_DEV_BAD_MASK of any of its rows) has NaN rows.  Ids that do not ascend,
 * lie outside [0, V) or have a negative count are reported (SV_DEV_BAD_HISTORY, SV_DEV_BAD_BIAS) but leave open
 * which of the request's logits the penalties and biases reach.
 * Results are the same from call to call.
 */
sv_status spec_logits(const void *logits, sv_dtype dtype, const int32_t *draft_tokens, const int32_t *num_drafts,
                      const int32_t *row_offsets, int32_t B, int32_t k_max, int32_t V, int32_t total_rows,
                      sv_logit_rules rules, void *out, void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGITS_H */
