"""The attention half of one decoder layer for a batch of many variants' tokens,
and what follows the last layer: the head and the draw of the next tokens.

"Serving Architecture" keeps one base in HBM for every variant of the delta
cache; this module runs the layer around its linears the same way: one fused
q/k/v projection and one output projection through bitdelta_linear_grouped,
and between them the rotated append to the paged cache, attention over it, and
the norms, whose weights a variant keeps for itself (BitDelta codes the
linears only).  Every call takes the whole batch at once, whatever variants
and sequences it mixes.

A base may be held in 8 bits (quantize_int8 of its rows): the tokens' rows are then
quantised in front of it and go through bitdelta_linear_int8.
"""
from __future__ import annotations

import torch

from . import attention, block_norm, kv_append, linear_grouped, linear_int8, quantize_int8, sample

__all__ = ["AttentionBlock", "OutputBlock"]


def _linear(x, variant_ids, layer):
    """(w bf16, signs, alpha), or (w int8, its scales, signs, alpha)."""
    if len(layer) == 3:
        return linear_grouped(x, variant_ids, *layer, per_matrix=False)
    return linear_int8(*quantize_int8(x), *layer, variant_ids=variant_ids, per_matrix=False)


class AttentionBlock:
    """qkv and out: (w_base bf16 [d_out, d_in], signs uint8 [V, d_out, d_in/8],
    alpha fp32 [V, d_out]) of the two projections, or (w_base int8 [d_out, d_in],
    w_scale fp32 [d_out], signs, alpha) over a base in 8 bits; the rows of qkv are
    those of q, k and v after one another, head by head.  post_weight (norm of the
    block's output) and next_weight (norm before the next block): [V, d], both
    [d] for every variant, or None.  inv_freq: fp64 [rotary / 2] on the device."""

    def __init__(self, qkv, out, n_heads, kv, inv_freq, *, post_weight=None, next_weight=None, scale=1.0, eps=1e-6,
                 interleaved=False):
        self.qkv, self.out, self.n_heads, self.kv, self.inv_freq = qkv, out, n_heads, kv, inv_freq
        self.post_weight, self.next_weight = post_weight, next_weight
        self.scale, self.eps, self.interleaved = scale, eps, interleaved
        rows = (n_heads + 2 * kv.n_kv_heads) * kv.head_dim
        if qkv[0].shape[0] != rows:
            raise ValueError(f"qkv must have {rows} rows for {n_heads} + 2 x {kv.n_kv_heads} heads of {kv.head_dim} "
                             f"(got {qkv[0].shape[0]})")
        if out[0].shape[1] != n_heads * kv.head_dim:
            raise ValueError(f"out must have {n_heads * kv.head_dim} columns (got {out[0].shape[1]})")

    def forward(self, x, residual, variant_ids, batch, gate=None, gate_act="none"):
        """x: the block's normalised input bf16 [T, d]; residual [T, d] bf16 or
        fp32, updated in place; variant_ids int32 [T]; batch: the PagedBatch of
        the T tokens.  Appends the tokens' keys and values to the cache and
        returns (the next block's normalised input or None, residual)."""
        kv, D = self.kv, self.kv.head_dim
        fused = _linear(x, variant_ids, self.qkv)
        q, k, v = (t.unflatten(1, (-1, D)) for t in
                   fused.split([self.n_heads * D, kv.n_kv_heads * D, kv.n_kv_heads * D], 1))
        q = kv_append(q, k, v, self.inv_freq, kv, batch, interleaved=self.interleaved)
        o = attention(q, kv, batch)
        y = _linear(o.flatten(1), variant_ids, self.out)
        residual, x = block_norm(residual, y, post_weight=self.post_weight, gate=gate, gate_act=gate_act, scale=self.scale,
                                 pre_weight=self.next_weight, variant_ids=variant_ids, eps=self.eps,
                                 residual_out=residual)
        return x, residual


class OutputBlock:
    """head: (int8 [vocab, d], fp32 [vocab]) as quantize_int8 gives them for the
    rows of the output embedding, which all variants share."""

    def __init__(self, head):
        self.weight, self.weight_scale = head

    def logits(self, x, rows=None):
        """fp32 [n, vocab] of the normalised rows x bf16 [T, d], or of those that
        rows (int64 [n]) names: the last token of each sequence."""
        if rows is not None:
            x = x.index_select(0, rows)
        return linear_int8(*quantize_int8(x), self.weight, self.weight_scale, out_dtype=torch.float32)

    def forward(self, x, u, rows=None, **settings):
        """(tokens int32 [n], logprobs fp32 [n]) drawn by the random numbers u
        fp32 [n]; settings as sample takes them."""
        return sample(self.logits(x, rows), u, **settings)
