"""Linears over a shared base held in 8 bits (include/bitdelta_int8.h): rows as
int8 numbers with one scale each, and the product of such rows with an int8
base and the 1-bit deltas of the tokens' variants.

Argument marshalling only, as in the rest of the binding.
"""
from __future__ import annotations

import contextlib

import torch

from . import BD_ALPHA_MATRIX, BD_ALPHA_ROW, BD_BF16, BD_F32, BD_OK, check, lib
from .decoder import _dense, _refuse, _rows, _stream

__all__ = ["quantize_int8", "linear_int8"]

_Tensor = torch.Tensor
_BF16, _F32, _I8, _U8, _I32 = torch.bfloat16, torch.float32, torch.int8, torch.uint8, torch.int32


def _on(dev):
    """Launches go to the current device: make it the tensors' own."""
    return contextlib.nullcontext() if torch.cuda.current_device() == dev else torch.cuda.device(dev)


def quantize_int8(x, *, out=None, scale_out=None):
    """int8 numbers and one fp32 scale for each row of x: scale = max |x| / 127,
    q = x / scale to the nearest whole number, ties to even (zeros where a row
    is zero; scale NaN where it holds a NaN or an infinity).

    x bf16 or fp32 [..., d], the rows of a 2-d x may be strided.  For activations
    a row is a token, for a weight [d_out, d_in] an output channel.  Returns
    (q int8 [..., d], scale fp32 [...])."""
    xt = x.dtype if isinstance(x, _Tensor) else None
    if xt is not _BF16 and xt is not _F32:
        raise TypeError("x must be a bfloat16 or float32 tensor")
    dev = x.get_device()
    if dev < 0 or x.dim() < 1:
        _refuse(x, xt, "x", (None, None), None)
    lead, d = x.shape[:-1], x.shape[-1]
    if x.dim() == 2:
        xp, xs = _rows(x, xt, "x", x.shape, dev)
        m = lead[0]
    else:
        xp, xs = _dense(x, xt, "x", x.shape, dev), d
        m = x.numel() // d if d else 0
    if out is None:
        out = torch.empty_like(x, dtype=_I8, memory_format=torch.contiguous_format)
        op = out.data_ptr()
    else:
        op = _dense(out, _I8, "out", x.shape, dev)
    if scale_out is None:
        scale_out = x.new_empty(lead, dtype=_F32)
        sp = scale_out.data_ptr()
    else:
        sp = _dense(scale_out, _F32, "scale_out", lead, dev)
    with _on(dev):
        status = lib.bitdelta_quantize_int8(xp, xs, BD_F32 if xt is _F32 else BD_BF16, m, d, op, sp, _stream(dev))
    if status:
        check(status)
    return out, scale_out


def linear_int8(q, q_scale, weight, weight_scale, delta_sign=None, alpha=None, *, variant_ids=None,
                per_matrix: bool | None = None, out_dtype=torch.bfloat16, out=None):
    """y = q_scale * (weight_scale * (q weight^T) + alpha * (q sign^T)), the sums
    exact, for tokens of one or many variants over one int8 base.

    q int8 [..., d_in] and q_scale fp32 [...] as quantize_int8 gives them for the
    activations, weight int8 [d_out, d_in] and weight_scale fp32 [d_out] as it
    gives them for the base.  delta_sign uint8 [d_out, d_in/8] with alpha fp32
    [d_out] or [1]: one delta for every token; None: no delta.  With variant_ids
    int32, one for each row of a 2-d q: delta_sign [V, d_out, d_in/8], alpha
    [V, d_out] or [V] (per_matrix); a token whose id is none of [0, V) gives a
    zero row.  Returns y [..., d_out] of out_dtype (bfloat16 or float32)."""
    dev = q.get_device() if isinstance(q, _Tensor) else -1
    if dev < 0 or q.dim() < 1:
        _refuse(q, _I8, "q", (None, None), None)
    if not isinstance(weight, _Tensor) or weight.dim() != 2:
        _refuse(weight, _I8, "weight", (None, q.shape[-1]), dev)
    lead, d_in = q.shape[:-1], q.shape[-1]
    d_out = weight.shape[0]
    m = 1
    for n in lead:
        m *= n
    qp = _dense(q, _I8, "q", q.shape, dev)
    sp = _dense(q_scale, _F32, "q_scale", lead, dev)
    wp = _dense(weight, _I8, "weight", (d_out, d_in), dev)
    cp = _dense(weight_scale, _F32, "weight_scale", (d_out,), dev)
    dp = ap = ip = variants = 0
    mode = BD_ALPHA_ROW
    if delta_sign is not None:
        variants = 1
        signs = (d_out, d_in // 8)
        if variant_ids is not None:
            if len(lead) != 1:
                raise ValueError("with variant_ids q must be [m, d_in]")
            ip = _dense(variant_ids, _I32, "variant_ids", (m,), dev)
            if not isinstance(delta_sign, _Tensor) or delta_sign.dim() != 3:
                _refuse(delta_sign, _U8, "delta_sign", (None, *signs), dev)
            variants = delta_sign.shape[0]
            signs = (variants, *signs)
        dp = _dense(delta_sign, _U8, "delta_sign", signs, dev)
        if not isinstance(alpha, _Tensor):
            raise TypeError("alpha must be a torch.Tensor")
        if per_matrix is None:
            per_matrix = alpha.dim() <= 1 and d_out != 1 and alpha.numel() == variants
        if per_matrix:
            mode = BD_ALPHA_MATRIX
        ap = _dense(alpha, _F32, "alpha", (variants,) if per_matrix else signs[:-1], dev)
    elif alpha is not None or variant_ids is not None:
        raise ValueError("alpha and variant_ids need a delta_sign")
    if out is None:
        if out_dtype is not _BF16 and out_dtype is not _F32:
            raise TypeError("out_dtype must be bfloat16 or float32")
        out = q.new_empty((*lead, d_out), dtype=out_dtype)
        op = out.data_ptr()
    else:
        out_dtype = out.dtype if isinstance(out, _Tensor) and out.dtype is _F32 else _BF16
        op = _dense(out, out_dtype, "out", (*lead, d_out), dev)
    nws = lib.bitdelta_linear_int8_workspace(m, variants, d_out, d_in)
    ws = q.new_empty((nws,), dtype=_U8) if nws else None
    with _on(dev):
        status = lib.bitdelta_linear_int8(qp, sp, m, wp, cp, dp, ap, mode, ip, variants, d_out, d_in, op,
                                          BD_F32 if out_dtype is _F32 else BD_BF16, ws.data_ptr() if nws else 0, nws,
                                          _stream(dev))
    if status != BD_OK:
        check(status)
    return out
