/*
 * bitdelta_int8.h -- C ABI of linears over a shared base held in 8 bits: rows
 * as int8 numbers with one scale each, and the product of such rows with an
 * int8 base (a scale per output channel) and the 1-bit deltas of the tokens'
 * variants.
 *
 * bitdelta.h's conventions hold (device pointers, no allocation, asynchronous
 * on `stream`, host-side checks before any launch, status codes, packed signs).
 */
#ifndef BITDELTA_INT8_H
#define BITDELTA_INT8_H

#include "bitdelta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------- quantize_int8
 * Row i of x (bf16 or fp32 [m, d], row stride x_stride >= d elements):
 *   scale[i] = fl32(max_j |x[i,j]| / 127)
 *   q[i,j]   = x[i,j] / scale[i] to the nearest whole number, ties to even,
 *              clamped to [-127, 127]
 * the quotient taken exactly.  Rows of zeros, and rows whose scale rounds to
 * zero (max below 2^-143), give scale 0 and zeros.  A row that holds a NaN or an
 * infinity gives scale NaN and zeros, so that it stays visible in what is
 * computed from it.  q: int8 [m, d] dense, scale: fp32 [m].  The same call
 * serves activations (rows are tokens) and weights (rows are output channels).
 * Element alignment is enough for x and q, which do not overlap.  1 <= d <= BD_INT8_MAX_WIDTH. */
#define BD_INT8_MAX_WIDTH 131064

BD_API bd_status bitdelta_quantize_int8(const void *x, int64_t x_stride, int x_dtype, int64_t m, int64_t d, int8_t *q,
                                 float *scale, void *stream);

/* ------------------------------------------------------------- linear_int8
 * Token i of m, variant v:
 *   A = sum_k q[i,k] w[r,k],   B = sum_k q[i,k] sign_v[r,k]     (exact, int32)
 *   y[i,r] = q_scale[i] * (w_scale[r] * A + alpha_v[r] * B)
 * in 64 bits, then rounded to fp32 and to y's type.  Unlike W_eff of
 * bitdelta_linear the sum of base and delta is not rounded to bf16 in between.
 *   signs NULL:       no delta (alpha NULL, variant_ids NULL); B = 0.
 *   variant_ids NULL: one delta for every token, n_variants = 1; signs
 *                     [d_out, d_in/8], alpha [d_out] or [1] by alpha_mode.
 *   variant_ids:      int32 [m]; signs [n_variants, d_out, d_in/8], alpha
 *                     [n_variants, d_out] or [n_variants].  A token whose id is
 *                     outside [0, n_variants) gets a zero row.
 * q: int8 [m, d_in], w: int8 [d_out, d_in], any of the 256 numbers; q_scale: fp32
 * [m], w_scale: fp32 [d_out]; y: [m, d_out] of y_dtype (BD_BF16 or BD_F32); all
 * dense, q and w 16-byte aligned, y 16-byte aligned, signs of any alignment.
 * d_in: a multiple of 8, at most BD_INT8_MAX_WIDTH; q, w, one variant's signs and y
 * each below 2 GiB.
 * workspace: at least bitdelta_linear_int8_workspace() bytes, 16-byte aligned,
 * scratch (n_variants as in the call, 0 without deltas); at most 2^29 bytes and what
 * a table of the tokens takes.  y and workspace overlap nothing else.  The result does not depend
 * on how a call is cut, nor on its other tokens: sums of whole numbers are exact in any order. */
BD_API size_t bitdelta_linear_int8_workspace(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in);
BD_API bd_status bitdelta_linear_int8(const int8_t *q, const float *q_scale, int64_t m, const int8_t *w,
                               const float *w_scale, const uint8_t *signs, const float *alpha, int alpha_mode,
                               const int32_t *variant_ids, int32_t n_variants, int64_t d_out, int64_t d_in,
                               void *y, int y_dtype, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BITDELTA_INT8_H */
