"""What stands between the linears of a served decoder layer
(include/bitdelta_decoder.h): block norms with per-variant weights, the append
of rotated keys and values to a paged cache, and attention over it.

Argument marshalling only, as in the rest of the binding.  PagedKV and
PagedBatch hold the tensors of a cache and of a batch together with the C
structs that describe them, so a call over many layers describes them once;
the tensors' contents are read by the kernels at each call.
"""
from __future__ import annotations

import ctypes

import torch

from . import BD_BF16, BD_F32, check, lib

__all__ = ["block_norm", "kv_append", "attention", "PagedKV", "PagedBatch"]

BD_KV_BF16, BD_KV_E4M3 = 0, 1
GATE_ACTS = {"none": 0, "sigmoid": 1, "silu": 2}

_VP = ctypes.c_void_p


class _KvCache(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP), ("k_scale", _VP), ("v_scale", _VP), ("dtype", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("q_start", _VP), ("kv_len", _VP), ("page_table", _VP), ("group_start", _VP), ("prefix_len", _VP),
                ("prefix_table", _VP), ("n_tokens", ctypes.c_int64), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("max_prefix_pages", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


_Tensor = torch.Tensor
_BF16, _F32, _I32, _F64, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float64, torch.float8_e4m3fn
# the raw handle alone: a torch.cuda.Stream object costs as much as the call itself
_stream = torch._C._cuda_getCurrentRawStream


def _refuse(t, dtype, name, shape, dev):
    """Say what is wrong with a tensor that a fast check has turned down.
    `shape` may hold None for a free extent; dev is a device index."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device (got {t.device})")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} (got {t.device})")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    raise ValueError(f"{name} must be contiguous (got strides {list(t.stride())})")


def _dense(t, dtype, name, shape, dev):
    """Address of a contiguous tensor."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, name, shape, dev)


def _like(t):
    """A contiguous tensor of t's shape and type (options cost as much as the allocation)."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _rows(t, dtype, name, shape, dev):
    """Address and row stride of an [m, d] tensor whose rows are dense."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        m, d = shape
        rs, cs = t.stride()
        if cs == 1 or d <= 1:
            # the stride of a single row is not used and may be anything
            if m <= 1:
                return t.data_ptr(), d
            if rs >= d:
                return t.data_ptr(), rs
        raise ValueError(f"{name} needs dense rows that do not overlap (got strides {[rs, cs]})")
    _refuse(t, dtype, name, shape, dev)


def _heads(t, name, shape, kv):
    """Address and token stride of a bf16 [T, H, head_dim] tensor whose heads are dense."""
    if isinstance(t, _Tensor) and t.dtype is _BF16 and t.dim() == 3 and t.get_device() == kv._dev:
        T, H, D = t.shape
        if D == kv.head_dim and shape[0] in (None, T) and shape[1] in (None, H):
            ts, hs, cs = t.stride()
            if cs == 1 and (hs == D or H <= 1):
                if T <= 1:
                    return t.data_ptr(), H * D
                if ts >= H * D:
                    return t.data_ptr(), ts
            raise ValueError(f"{name} must be dense but for its token stride (got strides {[ts, hs, cs]})")
    _refuse(t, _BF16, name, (*shape, kv.head_dim), kv._dev)


def block_norm(residual, block=None, *, post_weight=None, gate=None, gate_act: str = "none", scale: float = 1.0,
               pre_weight=None, variant_ids=None, eps: float = 1e-6, residual_out=None, out=None):
    """r' = residual + scale * act(gate) * rms(block) * post_weight[v] and
    x = rms(r') * pre_weight[v], v = variant_ids[token].

    residual bf16 or fp32 [m, d]; block, gate bf16 [m, d]; weights bf16 or
    fp32 (both the same) [V, d], or [d] for every variant; variant_ids int32
    [m] (needed where V > 1; they pick nothing where the weights are [d] or
    None).  Rows may be strided.  block None: no update; post_weight None: the
    block is added as it is; pre_weight None: no x.  residual_out may be
    residual (in place); None allocates it where there is a block.  Returns
    (r', x): r' is `residual` without a block, x None without pre_weight."""
    rt = residual.dtype if isinstance(residual, _Tensor) else None
    if rt is not _BF16 and rt is not _F32:
        raise TypeError("residual must be a bfloat16 or float32 tensor")
    dev, shape = residual.get_device(), residual.shape
    if dev < 0 or len(shape) != 2:
        _refuse(residual, rt, "residual", (None, None), None)
    rp, rs = _rows(residual, rt, "residual", shape, dev)
    m, d = shape
    act = GATE_ACTS.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACTS)}")
    bp = gp = bs = gs = 0
    if block is not None:
        bp, bs = _rows(block, _BF16, "block", shape, dev)
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate need a block")
    if gate is not None:
        gp, gs = _rows(gate, _BF16, "gate", shape, dev)
    weight = post_weight if pre_weight is None else pre_weight
    wt, n_variants, post, pre = 0, 1, 0, 0
    if weight is not None:
        dtype = weight.dtype if isinstance(weight, _Tensor) else None
        if dtype is not _BF16 and dtype is not _F32:
            raise TypeError("weights must be bfloat16 or float32 tensors")
        want = weight.shape
        wt = BD_F32 if dtype is _F32 else BD_BF16
        if not 1 <= len(want) <= 2 or want[-1] != d or want[0] < 1:
            raise ValueError(f"weights must be [V, {d}] or [{d}] (got {list(want)})")
        n_variants = want[0] if len(want) == 2 else 1
        if post_weight is not None:
            post = _dense(post_weight, dtype, "post_weight", want, dev)
        if pre_weight is not None:
            pre = _dense(pre_weight, dtype, "pre_weight", want, dev)
    ids = 0
    if variant_ids is not None:
        ids = _dense(variant_ids, _I32, "variant_ids", (m,), dev)
        if weight is None or weight.dim() == 1:
            ids = 0        # nothing to pick: no weight, or one for every variant
    elif n_variants > 1:
        raise ValueError("weights of several variants need variant_ids")
    op = os = xp = 0
    if residual_out is not None:
        op, os = _rows(residual_out, rt, "residual_out", shape, dev)
    elif block is not None:
        residual_out = _like(residual)
        op, os = residual_out.data_ptr(), d
    if pre_weight is not None:
        if out is None:
            like = residual if rt is _BF16 else block
            out = _like(like) if like is not None else torch.empty_like(residual, dtype=_BF16,
                                                                        memory_format=torch.contiguous_format)
            xp = out.data_ptr()
        else:
            xp = _dense(out, _BF16, "out", shape, dev)
    elif out is not None:
        raise ValueError("out needs a pre_weight")
    status = lib.bitdelta_block_norm(rp, rs, BD_F32 if rt is _F32 else BD_BF16, bp, bs, gp, gs, act, scale, post, pre, wt,
                                     ids, n_variants, m, d, eps, op, os, xp, _stream(dev))
    if status:
        check(status)
    return (residual if residual_out is None else residual_out), out


class PagedKV:
    """A paged key / value cache: k and v [n_pages, n_kv_heads, page_size,
    head_dim], bf16 or float8_e4m3fn (a stored number stands for number *
    scale[head], scales fp32 [n_kv_heads], None = 1)."""

    def __init__(self, k, v, *, k_scale=None, v_scale=None):
        if not isinstance(k, _Tensor) or k.dtype not in (_BF16, _E4M3):
            raise TypeError("k must be a bfloat16 or float8_e4m3fn tensor")
        if not k.is_cuda or k.dim() != 4:
            _refuse(k, k.dtype, "k", (None, None, None, None), None)
        dev = k.get_device()
        kp = _dense(k, k.dtype, "k", k.shape, dev)
        vp = _dense(v, k.dtype, "v", k.shape, dev)
        e4m3 = k.dtype is _E4M3
        if not e4m3 and (k_scale is not None or v_scale is not None):
            raise ValueError("a bf16 cache takes no scales")
        sp = [0 if s is None else _dense(s, _F32, n, (k.shape[1],), dev)
              for s, n in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self._dev = k.device, dev
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self._c = _KvCache(kp, vp, sp[0], sp[1], BD_KV_E4M3 if e4m3 else BD_KV_BF16, *k.shape)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, n_pages, n_kv_heads, page_size, head_dim, dtype=torch.bfloat16, device=None, **scales):
        """A cache of unwritten pages."""
        dev = torch.device("cuda") if device is None else device
        k, v = (torch.empty((n_pages, n_kv_heads, page_size, head_dim), dtype=dtype, device=dev) for _ in range(2))
        return cls(k, v, **scales)


class PagedBatch:
    """The sequences of a call over a paged cache (bd_batch in
    include/bitdelta_decoder.h).  q_start int32 [n_seqs + 1], kv_len int32
    [n_seqs] (new tokens included), page_table int32 [n_seqs, max_pages];
    with prefixes shared by neighbouring sequences group_start int32
    [n_groups + 1], prefix_len int32 [n_groups] and prefix_table int32
    [n_groups, max_prefix_pages].  max_new: the largest number of new tokens of
    a sequence, 0 = unknown (a hint).  The tensors may be rewritten in place
    between calls."""

    def __init__(self, q_start, kv_len, page_table, *, group_start=None, prefix_len=None, prefix_table=None,
                 max_new: int = 0):
        for t, name, dim in ((kv_len, "kv_len", 1), (page_table, "page_table", 2)):
            if not isinstance(t, _Tensor) or t.dtype is not _I32 or not t.is_cuda or t.dim() != dim:
                _refuse(t, _I32, name, (None,) * dim, None)
        dev, n = kv_len.get_device(), kv_len.shape[0]
        ptrs = [_dense(q_start, _I32, "q_start", (n + 1,), dev), _dense(kv_len, _I32, "kv_len", (n,), dev),
                _dense(page_table, _I32, "page_table", (n, page_table.shape[1]), dev), 0, 0, 0]
        groups = prefix_pages = 0
        given = [t is not None for t in (group_start, prefix_len, prefix_table)]
        if any(given):
            if not all(given):
                raise ValueError("group_start, prefix_len and prefix_table come together")
            for t, name, dim in ((prefix_len, "prefix_len", 1), (prefix_table, "prefix_table", 2)):
                if not isinstance(t, _Tensor) or t.dtype is not _I32 or t.dim() != dim:
                    _refuse(t, _I32, name, (None,) * dim, dev)
            groups, prefix_pages = prefix_len.shape[0], prefix_table.shape[1]
            ptrs[3:] = [_dense(group_start, _I32, "group_start", (groups + 1,), dev),
                        _dense(prefix_len, _I32, "prefix_len", (groups,), dev),
                        _dense(prefix_table, _I32, "prefix_table", (groups, prefix_pages), dev)]
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.group_start, self.prefix_len, self.prefix_table = group_start, prefix_len, prefix_table
        self.device, self._dev = kv_len.device, dev
        # n_tokens is each call's own: one struct for every number of tokens seen
        self._fields = (*ptrs, 0, n, page_table.shape[1], groups, prefix_pages, int(max_new))
        self._by_tokens = {}

    def _struct(self, n_tokens, kv):
        if self._dev != kv._dev:
            raise ValueError(f"the batch is on {self.device}, the cache on {kv.device}")
        held = self._by_tokens.get(n_tokens)
        if held is None:
            c = _Batch(*self._fields[:6], n_tokens, *self._fields[7:])
            held = self._by_tokens[n_tokens] = (ctypes.addressof(c), c)
        return held[0]


def kv_append(q, k, v, inv_freq, kv: PagedKV, batch: PagedBatch, *, interleaved: bool = False, q_out=None):
    """Rotate q and k by their positions and store k and v at their places of
    the cache.  q bf16 [T, H, D] (or None), k and v bf16 [T, H_kv, D], token
    strides free (views of a fused projection); inv_freq fp64 [rotary / 2] in
    radians a position (None: no rotation).  Returns the rotated q: a new
    tensor, or q_out where given (which may be q itself where it is dense)."""
    kp, ks = _heads(k, "k", (None, kv.n_kv_heads), kv)
    T = k.shape[0]
    vp, vs = _heads(v, "v", (T, kv.n_kv_heads), kv)
    qp = qs = H = op = fp = rotary = 0
    if q is not None:
        qp, qs = _heads(q, "q", (T, None), kv)
        H = q.shape[1]
        if q_out is None:
            q_out = _like(q)
            op = q_out.data_ptr()
        else:
            op = _dense(q_out, _BF16, "q_out", q.shape, kv._dev)
    elif q_out is not None:
        raise ValueError("q_out needs a q")
    if inv_freq is not None:
        if not isinstance(inv_freq, _Tensor) or inv_freq.dim() != 1:
            _refuse(inv_freq, _F64, "inv_freq", (None,), kv._dev)
        fp = _dense(inv_freq, _F64, "inv_freq", inv_freq.shape, kv._dev)
        rotary = 2 * inv_freq.shape[0]
    status = lib.bitdelta_kv_append(qp, qs, kp, ks, vp, vs, H, fp, rotary, 1 if interleaved else 0, kv._ref,
                                    batch._struct(T, kv), op, _stream(kv._dev))
    if status:
        check(status)
    return q_out


def attention(q, kv: PagedKV, batch: PagedBatch, *, scale: float | None = None, out=None):
    """Causal attention of the batch's new tokens over the cache (their own
    keys appended before), every group's prefix included.  q bf16 [T, H, D],
    token stride free; scale: D ** -0.5 by default.  Returns out bf16
    [T, H, D]; padding tokens and tokens that see no key give zero rows."""
    qp, qs = _heads(q, "q", (None, None), kv)
    T, H, D = q.shape
    if out is None:
        out = _like(q)
        op = out.data_ptr()
    else:
        op = _dense(out, _BF16, "out", q.shape, kv._dev)
    b = batch._struct(T, kv)
    nws = lib.bitdelta_attention_workspace(H, kv._ref, b)
    ws = torch.empty((nws,), dtype=torch.uint8, device=kv.device) if nws else None
    status = lib.bitdelta_attention(qp, qs, H, D ** -0.5 if scale is None else scale, kv._ref, b, op,
                                    ws.data_ptr() if nws else 0, nws, _stream(kv._dev))
    if status:
        check(status)
    return out
