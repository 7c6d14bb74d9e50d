"""The draw of next tokens from logits (include/bitdelta_sample.h).

Argument marshalling only, as in the rest of the binding.
"""
from __future__ import annotations

import torch

from . import BD_BF16, BD_F32, check, lib
from .decoder import _BF16, _F32, _I32, _Tensor, _dense, _refuse, _rows, _stream
from .int8 import _on

__all__ = ["sample"]


def _each(value, dtype, name, m, dev):
    """(address or 0, value for all rows) of a setting: a tensor of one value a row, or a number."""
    if isinstance(value, _Tensor):
        return _dense(value, dtype, name, (m,), dev), 0
    if isinstance(value, bool) or not isinstance(value, (int, float)):
        raise TypeError(f"{name} must be a torch.Tensor or a number")
    if dtype is not _I32:
        return 0, float(value)
    if not isinstance(value, int) or value >= 2 ** 31:
        raise TypeError(f"{name} must be a whole number below 2^31")
    return 0, max(value, 0)


def sample(logits, u, *, temperature=1.0, top_k=None, top_p=None, min_p=None, out=None, logprobs_out=None):
    """Draw one token from every row of logits by the given random numbers.

    logits bf16 or fp32 [m, vocab] (rows may be strided), u fp32 [m] in [0, 1).
    temperature, top_p, min_p (fp32 [m]) and top_k (int32 [m]) are one value a row
    or a number for all of them; None, and top_k <= 0, top_p >= 1, min_p <= 0: no
    limit.  temperature <= 0 takes the largest logit.

    In the order of the logits, largest first and equal ones by index: top_k keeps
    the first k, top_p of those each token in front of which less than top_p of
    their probability lies, min_p the tokens at least min_p as probable as the
    first; the token drawn is the first whose running sum passes u times the sum
    of what is kept.  Tokens of -inf (or NaN) are never drawn.

    Returns (tokens int32 [m], logprobs fp32 [m]), the logarithm of the probability
    with which each token was drawn; (-1, -inf) for a row without a token to draw."""
    dtype = logits.dtype if isinstance(logits, _Tensor) else None
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError("logits must be a bfloat16 or float32 tensor")
    dev, shape = logits.get_device(), logits.shape
    if dev < 0 or len(shape) != 2:
        _refuse(logits, dtype, "logits", (None, None), None)
    lp, ls = _rows(logits, dtype, "logits", shape, dev)
    m, vocab = shape
    up = _dense(u, _F32, "u", (m,), dev)
    tp, t = _each(1.0 if temperature is None else temperature, _F32, "temperature", m, dev)
    kp, k = _each(0 if top_k is None else top_k, _I32, "top_k", m, dev)
    pp, p = _each(1.0 if top_p is None else top_p, _F32, "top_p", m, dev)
    np_, n = _each(0.0 if min_p is None else min_p, _F32, "min_p", m, dev)
    if out is None:
        out = logits.new_empty((m,), dtype=_I32)
        op = out.data_ptr()
    else:
        op = _dense(out, _I32, "out", (m,), dev)
    if logprobs_out is None:
        logprobs_out = logits.new_empty((m,), dtype=_F32)
        gp = logprobs_out.data_ptr()
    else:
        gp = _dense(logprobs_out, _F32, "logprobs_out", (m,), dev)
    nws = lib.bitdelta_sample_workspace(m, vocab)
    ws = logits.new_empty((nws,), dtype=torch.uint8) if nws else None
    with _on(dev):
        status = lib.bitdelta_sample(lp, ls, BD_F32 if dtype is _F32 else BD_BF16, m, vocab, up, tp, t, kp, k, pp, p, np_, n,
                                     op, gp, ws.data_ptr() if nws else 0, nws, _stream(dev))
    if status:
        check(status)
    return out, logprobs_out
