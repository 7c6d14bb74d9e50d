/*
 * bitdelta_sample.h -- C ABI of the draw of next tokens from logits.
 *
 * bitdelta.h's conventions hold (device pointers, no allocation, asynchronous
 * on `stream`, host-side checks before any launch, status codes).
 */
#ifndef BITDELTA_SAMPLE_H
#define BITDELTA_SAMPLE_H

#include "bitdelta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ sample
 * Row i of m.  The tokens stand in the order of their logits, largest first,
 * equal ones by their index; weights w_j = exp((l_j - l_0) / temperature) in
 * that order, sums C_j = w_0 + ... + w_j.  The limits each keep a beginning of it:
 *   top_k   the first top_k tokens (all where top_k <= 0)
 *   top_p   of those, token j while C_{j-1} < top_p * C of what top_k left
 *           (no limit where top_p >= 1 or NaN)
 *   min_p   token j while w_j >= min_p (no limit where min_p <= 0 or NaN)
 * and the first token is always kept.  With n tokens kept the token drawn is the
 * first with C_j > u * C_{n-1}; logprob = ln(w_j / C_{n-1}), the probability with
 * which it was drawn.  temperature <= 0 or NaN: the first token, logprob 0; +inf:
 * all tokens alike.  u below 0 or NaN counts as 0; from 1 on the last kept token
 * with a weight is drawn.
 * A logit of -inf or NaN is never drawn; one of +inf has weight 1 and leaves the
 * others none.  A row without a token that can be drawn gives token -1 and
 * logprob -inf.
 * Weights are held to within 2^-37 of themselves, in whole numbers whose sums are
 * exact, so the result does not depend on how a row is cut; a token below exp(-32)
 * of the first may count as one without weight.  logprob is formed from what is
 * kept beside the token drawn: near 0 it is right to about 2^-35 of itself, and 0
 * where the token is kept alone.
 * logits: [m, vocab] of logits_dtype (BD_BF16 or BD_F32), row stride in elements
 * (>= vocab), element alignment; u: fp32 [m]; temperature, top_p, min_p fp32 [m],
 * top_k int32 [m], each NULL for the call's one value *_all.  tokens: int32 [m],
 * logprobs: fp32 [m] or NULL.
 * 1 <= vocab <= BD_SAMPLE_MAX_VOCAB, m <= BD_SAMPLE_MAX_ROWS (BD_ESHAPE otherwise).  workspace: at least
 * bitdelta_sample_workspace() bytes, 16-byte aligned, scratch; little more than 2^28
 * bytes at most.  Outputs and workspace overlap nothing else. */
#define BD_SAMPLE_MAX_VOCAB 1048576
#define BD_SAMPLE_MAX_ROWS 131072

BD_API size_t bitdelta_sample_workspace(int64_t m, int64_t vocab);
BD_API bd_status bitdelta_sample(const void *logits, int64_t logits_stride, int logits_dtype, int64_t m, int64_t vocab,
                          const float *u, const float *temperature, float temperature_all,
                          const int32_t *top_k, int32_t top_k_all, const float *top_p, float top_p_all,
                          const float *min_p, float min_p_all, int32_t *tokens, float *logprobs,
                          void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BITDELTA_SAMPLE_H */
