/*
 * bitdelta_decoder.h -- C ABI of what stands between the linears of a served
 * decoder layer: block norms with per-variant weights, the append of rotated
 * keys and values to a paged cache, and causal attention over that cache with
 * prefixes shared by several sequences of the batch.
 *
 * bitdelta.h's conventions hold (device pointers, no allocation, asynchronous
 * on `stream`, host-side checks before any launch, status codes).  What the
 * device holds in its integer arrays (variant ids, starts, lengths, page
 * numbers) cannot be checked on the host; the kernels bound every such value
 * themselves, as stated per field, and never address outside the buffers that
 * a call describes.
 */
#ifndef BITDELTA_DECODER_H
#define BITDELTA_DECODER_H

#include "bitdelta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------------------------------- block_norm
 * Token i of m, variant v = variant_ids[i] (v = 0 where variant_ids is NULL):
 *   y   = block[i] * rsqrt(mean_j(block[i,j]^2) + eps) * post_weight[v]
 *   r'  = residual[i] + scale * act(gate[i]) * y
 *   x   = bf16(r' * rsqrt(mean_j(r'[j]^2) + eps) * pre_weight[v])
 * in fp32, each output rounded once (the second norm reads r' before its
 * rounding).
 *   block NULL: r' = residual (no post_weight and no gate then).
 *   post_weight NULL: y = block.     gate NULL: act(gate) = 1.
 *   pre_weight NULL: x is not written (and may be NULL).
 *   residual_out NULL: r' is not written; it may be residual itself (same
 *     stride), and aliases nothing else.
 * residual, residual_out: [m, d] of residual_dtype (BD_BF16 or BD_F32); block,
 * gate: bf16 [m, d]; each with its own row stride in elements (>= d); x: bf16
 * [m, d], dense.  post_weight, pre_weight: [n_variants, d] of weight_dtype, dense.
 * A token whose id is outside [0, n_variants) gets a zero row of x and
 * r' = residual.  With neither weight the ids pick nothing and are not read.
 * Element alignment is enough; rows that start on 16 bytes load fastest.
 * 1 <= d <= BD_NORM_MAX_WIDTH (BD_ESHAPE otherwise). */
#define BD_NORM_MAX_WIDTH 32768

typedef enum { BD_GATE_NONE = 0, BD_GATE_SIGMOID = 1, BD_GATE_SILU = 2 } bd_gate_act;

BD_API bd_status bitdelta_block_norm(const void *residual, int64_t residual_stride, int residual_dtype,
                              const bd_bf16 *block, int64_t block_stride,
                              const bd_bf16 *gate, int64_t gate_stride, int gate_act, float scale,
                              const void *post_weight, const void *pre_weight, int weight_dtype,
                              const int32_t *variant_ids, int32_t n_variants,
                              int64_t m, int64_t d, float eps,
                              void *residual_out, int64_t residual_out_stride, bd_bf16 *x, void *stream);

/* ------------------------------------------------------------- paged cache
 * k and v: [n_pages, n_kv_heads, page_size, head_dim], dense, 16-byte aligned.
 * page_size: a power of two in [1, 1024]; head_dim: 64 or 128; n_kv_heads at
 * most 1024; n_pages * n_kv_heads * page_size below 2^31.
 * dtype BD_KV_E4M3: a stored number stands for number * scale[head], with
 * k_scale / v_scale fp32 [n_kv_heads] (NULL: 1), of any sign or zero (an
 * append divides by them: by zero it stores +-448, and NaN for a zero);
 * BD_KV_BF16 takes no scales. */
typedef enum { BD_KV_BF16 = 0, BD_KV_E4M3 = 1 } bd_kv_dtype;

typedef struct {
    void *k, *v;
    const float *k_scale, *v_scale;
    int32_t dtype;
    int32_t n_pages, n_kv_heads, page_size, head_dim;
} bd_kv_cache;

/* -------------------------------------------------------------- the batch
 * Sequence s owns the tokens [q_start[s], q_start[s+1]) of the call's
 * n_tokens; q_start (int32 [n_seqs+1]) does not decrease.  Tokens that belong
 * to no sequence are padding.  kv_len[s] (int32) counts the keys in the
 * sequence's own pages with the new tokens included, so new token i of n has
 * place kv_len[s] - n + i there, and sees the places up to its own.  Place p
 * is slot p % page_size of page page_table[s, p / page_size] (int32
 * [n_seqs, max_pages]).
 * A group g of neighbouring sequences [group_start[g], group_start[g+1])
 * (int32 [n_groups+1], not decreasing) stands behind a common prefix of
 * prefix_len[g] keys in the pages prefix_table[g, :] (int32 [n_groups,
 * max_prefix_pages]): every token of the group sees all of them, and its
 * position is prefix_len[g] + its place.  n_groups = 0: no prefixes, the
 * three pointers may be NULL.  n_seqs = 0: padding alone, the three pointers
 * of the sequences may be NULL, with groups or without.
 * Bounds kept on the device: starts are clamped to [0, n_tokens], lengths to
 * what the table's columns hold and to 2^30; a place below 0 or a page number outside
 * [0, n_pages) holds no key (nothing is stored there and attention passes it
 * over).
 * max_new: the largest number of new tokens of one sequence, or 0 where the
 * caller does not know it; a hint for the choice of kernels, right or wrong: by
 * it the keys are summed in another order, and results agree within their
 * roundings.  n_seqs <= BD_MAX_SEQS, n_groups <= BD_MAX_GROUPS; n_tokens < 2^31, and
 * n_tokens * n_heads < 2^31 in the calls that take queries. */
#define BD_MAX_SEQS 4096
#define BD_MAX_GROUPS 256

typedef struct {
    const int32_t *q_start, *kv_len, *page_table;
    const int32_t *group_start, *prefix_len, *prefix_table;
    int64_t n_tokens;
    int32_t n_seqs, max_pages, n_groups, max_prefix_pages;
    int32_t max_new;
} bd_batch;

/* --------------------------------------------------------------- kv_append
 * Rotates q and k by their positions and stores k and v at their places.
 * With rotary = 2h and pos as above, pair i < h of a head turns by the angle
 * pos * inv_freq[i] (inv_freq fp64 [h]; the angle is reduced in fp64):
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * where the pair is columns (i, i + h), or (2i, 2i + 1) with `interleaved`;
 * columns from `rotary` on pass through.  rotary: a multiple of 16 in
 * [0, head_dim].  e4m3 cells are round-to-nearest-even of value / scale,
 * clamped to +-448 (NaN stays NaN).
 * q: bf16 [n_tokens, n_heads, head_dim] and k, v: bf16 [n_tokens, n_kv_heads,
 * head_dim] with token strides in elements (a multiple of 8), heads dense;
 * q_out: bf16 [n_tokens, n_heads, head_dim] dense; padding tokens and tokens
 * at a place below 0 give zero rows.  q and q_out NULL with n_heads = 0: no
 * queries.  q_out may be q where q is dense. */
BD_API bd_status bitdelta_kv_append(const bd_bf16 *q, int64_t q_stride, const bd_bf16 *k, int64_t k_stride,
                             const bd_bf16 *v, int64_t v_stride, int32_t n_heads,
                             const double *inv_freq, int32_t rotary, int interleaved,
                             const bd_kv_cache *cache, const bd_batch *batch, bd_bf16 *q_out, void *stream);

/* --------------------------------------------------------------- attention
 * out[t, h] = sum_j softmax_j(scale * q[t, h] . k[j, h / G]) v[j, h / G] over
 * the keys j that token t sees (the prefix of its group, then its own places
 * up to its own), G = n_heads / n_kv_heads whole.  fp32 scores and sums, the
 * weights enter the second product in bf16, the output is rounded once.
 * A token that sees no key, and a padding token, gives a zero row, and so does
 * one all of whose scores are -inf.  Cells that no token sees may hold anything,
 * NaN included; what is not finite in a key or value goes into the sums of the
 * tokens that see it, as the formula has it, and into no others.
 * q: bf16 [n_tokens, n_heads, head_dim], token stride in elements (a multiple
 * of 8), heads dense; out: the same, dense; q and out 16-byte aligned.
 * workspace: at least bitdelta_attention_workspace() bytes, 16-byte aligned,
 * scratch.  The query reads the host fields of batch and cache only. */
BD_API size_t bitdelta_attention_workspace(int32_t n_heads, const bd_kv_cache *cache, const bd_batch *batch);
BD_API bd_status bitdelta_attention(const bd_bf16 *q, int64_t q_stride, int32_t n_heads, float scale,
                             const bd_kv_cache *cache, const bd_batch *batch, bd_bf16 *out,
                             void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BITDELTA_DECODER_H */
