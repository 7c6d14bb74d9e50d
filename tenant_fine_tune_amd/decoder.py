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


def _check(t, dtype, name, dim, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device (got {t.device})")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev} (got {t.device})")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions (got {t.dim()})")


def _dense(t, dtype, name, shape, dev):
    _check(t, dtype, name, len(shape), dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _rows(t, dtype, name, shape, dev):
    """Pointer and row stride of a [m, d] tensor whose rows are dense."""
    _check(t, dtype, name, 2, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    return t.data_ptr(), _row_stride(t, name, shape[1])


def _row_stride(t, name, width):
    m, d = t.shape[0], t.shape[-1]
    inner = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != inner:
            raise ValueError(f"{name} must be dense but for its first stride")
        inner *= size
    # a stride of a single row is not used and may be anything
    stride = t.stride(0) if m > 1 else width
    if stride < width:
        raise ValueError(f"{name} rows overlap")
    return stride


def block_norm(residual, block=None, *, post_weight=None, gate=None, gate_act: str = "none", scale: float = 1.0,
               pre_weight=None, variant_ids=None, eps: float = 1e-6, residual_out=None, out=None):
    """r' = residual + scale * act(gate) * rms(block) * post_weight[v] and
    x = rms(r') * pre_weight[v], v = variant_ids[token].

    residual bf16 or fp32 [m, d]; block, gate bf16 [m, d]; weights bf16 or
    fp32 (both the same) [V, d] or [d]; variant_ids int32 [m] (needed where
    V > 1).  Rows may be strided.  block None: no update; post_weight None: the
    block is added as it is; pre_weight None: no x.  residual_out may be
    residual (in place); None allocates it where there is a block.  Returns
    (r', x): r' is `residual` without a block, x None without pre_weight."""
    if not isinstance(residual, torch.Tensor) or residual.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("residual must be a bfloat16 or float32 tensor")
    _check(residual, residual.dtype, "residual", 2)
    dev, shape = residual.device, residual.shape
    m, d = shape
    rs = _row_stride(residual, "residual", d)
    if gate_act not in GATE_ACTS:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACTS)}")
    bp = gp = bs = gs = 0
    if block is not None:
        bp, bs = _rows(block, torch.bfloat16, "block", shape, dev)
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate need a block")
    if gate is not None:
        gp, gs = _rows(gate, torch.bfloat16, "gate", shape, dev)
    weight = pre_weight if pre_weight is not None else post_weight
    wt, n_variants, post, pre = torch.bfloat16, 1, 0, 0
    if weight is not None:
        wt = weight.dtype
        if wt not in (torch.bfloat16, torch.float32):
            raise TypeError("weights must be bfloat16 or float32")
        n_variants = weight.shape[0] if weight.dim() == 2 else 1
        want = (n_variants, d) if weight.dim() == 2 else (d,)
        if n_variants < 1:
            raise ValueError("weights must hold at least one variant")
        if post_weight is not None:
            post = _dense(post_weight, wt, "post_weight", want, dev)
        if pre_weight is not None:
            pre = _dense(pre_weight, wt, "pre_weight", want, dev)
    ids = 0
    if variant_ids is not None:
        ids = _dense(variant_ids, torch.int32, "variant_ids", (m,), dev)
    elif n_variants > 1:
        raise ValueError("weights of several variants need variant_ids")
    op = os = xp = 0
    if residual_out is not None:
        op, os = _rows(residual_out, residual.dtype, "residual_out", shape, dev)
    elif block is not None:
        residual_out = torch.empty(shape, dtype=residual.dtype, device=dev)
        op, os = residual_out.data_ptr(), d
    if pre_weight is not None:
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
            xp = out.data_ptr()
        else:
            xp = _dense(out, torch.bfloat16, "out", shape, dev)
    elif out is not None:
        raise ValueError("out needs a pre_weight")
    check(lib.bitdelta_block_norm(residual.data_ptr(), rs, BD_F32 if residual.dtype == torch.float32 else BD_BF16, bp,
                                  bs, gp, gs, GATE_ACTS[gate_act], scale, post, pre,
                                  BD_F32 if wt == torch.float32 else BD_BF16, ids, n_variants, m, d, eps, op, os, xp,
                                  _stream(dev)))
    return (residual if residual_out is None else residual_out), out


class PagedKV:
    """A paged key / value cache: k and v [n_pages, n_kv_heads, page_size,
    head_dim], bf16 or float8_e4m3fn (a stored number stands for number *
    scale[head], scales fp32 [n_kv_heads], None = 1)."""

    def __init__(self, k, v, *, k_scale=None, v_scale=None):
        if not isinstance(k, torch.Tensor) or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError("k must be a bfloat16 or float8_e4m3fn tensor")
        _check(k, k.dtype, "k", 4)
        kp = _dense(k, k.dtype, "k", k.shape, k.device)
        vp = _dense(v, k.dtype, "v", k.shape, k.device)
        e4m3 = k.dtype == torch.float8_e4m3fn
        if not e4m3 and (k_scale is not None or v_scale is not None):
            raise ValueError("a bf16 cache takes no scales")
        sp = [0 if s is None else _dense(s, torch.float32, n, (k.shape[1],), k.device)
              for s, n in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
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
        _check(kv_len, torch.int32, "kv_len", 1)
        dev, n = kv_len.device, kv_len.shape[0]
        _check(page_table, torch.int32, "page_table", 2, dev)
        ptrs = [_dense(q_start, torch.int32, "q_start", (n + 1,), dev),
                _dense(kv_len, torch.int32, "kv_len", (n,), dev),
                _dense(page_table, torch.int32, "page_table", (n, page_table.shape[1]), dev), 0, 0, 0]
        groups = prefix_pages = 0
        given = [t is not None for t in (group_start, prefix_len, prefix_table)]
        if any(given):
            if not all(given):
                raise ValueError("group_start, prefix_len and prefix_table come together")
            _check(prefix_len, torch.int32, "prefix_len", 1, dev)
            _check(prefix_table, torch.int32, "prefix_table", 2, dev)
            groups, prefix_pages = prefix_len.shape[0], prefix_table.shape[1]
            ptrs[3:] = [_dense(group_start, torch.int32, "group_start", (groups + 1,), dev),
                        _dense(prefix_len, torch.int32, "prefix_len", (groups,), dev),
                        _dense(prefix_table, torch.int32, "prefix_table", (groups, prefix_pages), dev)]
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.group_start, self.prefix_len, self.prefix_table = group_start, prefix_len, prefix_table
        self.device = dev
        # n_tokens is each call's own: one struct for every number of tokens seen
        self._fields = (*ptrs, 0, n, page_table.shape[1], groups, prefix_pages, int(max_new))
        self._by_tokens = {}

    def _struct(self, n_tokens):
        c = self._by_tokens.get(n_tokens)
        if c is None:
            f = self._fields
            c = self._by_tokens[n_tokens] = _Batch(*f[:6], n_tokens, *f[7:])
        return ctypes.addressof(c)


def _heads(t, name, kv, n_tokens=None, heads=None):
    """Pointer and token stride of a [T, H, head_dim] tensor whose heads are dense."""
    _check(t, torch.bfloat16, name, 3, kv.device)
    T, H, D = t.shape
    if D != kv.head_dim or (n_tokens is not None and T != n_tokens) or (heads is not None and H != heads):
        raise ValueError(f"{name} must be [{'T' if n_tokens is None else n_tokens}, "
                         f"{'H' if heads is None else heads}, {kv.head_dim}] (got {list(t.shape)})")
    return t.data_ptr(), _row_stride(t, name, H * D)


def _same_device(kv, batch):
    if batch.device != kv.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {kv.device}")


def kv_append(q, k, v, inv_freq, kv: PagedKV, batch: PagedBatch, *, interleaved: bool = False, q_out=None):
    """Rotate q and k by their positions and store k and v at their places of
    the cache.  q bf16 [T, H, D] (or None), k and v bf16 [T, H_kv, D], token
    strides free (views of a fused projection); inv_freq fp64 [rotary / 2] in
    radians a position (None: no rotation).  Returns the rotated q (q_out
    where given; q itself where it is dense: in place)."""
    _same_device(kv, batch)
    kp, ks = _heads(k, "k", kv, heads=kv.n_kv_heads)
    T = k.shape[0]
    vp, vs = _heads(v, "v", kv, T, kv.n_kv_heads)
    qp = qs = H = op = fp = rotary = 0
    if q is not None:
        qp, qs = _heads(q, "q", kv, T)
        H = q.shape[1]
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=kv.device)
            op = q_out.data_ptr()
        else:
            op = _dense(q_out, torch.bfloat16, "q_out", q.shape, kv.device)
    elif q_out is not None:
        raise ValueError("q_out needs a q")
    if inv_freq is not None:
        _check(inv_freq, torch.float64, "inv_freq", 1, kv.device)
        rotary = 2 * inv_freq.shape[0]
        fp = _dense(inv_freq, torch.float64, "inv_freq", inv_freq.shape, kv.device)
    check(lib.bitdelta_kv_append(qp, qs, kp, ks, vp, vs, H, fp, rotary, 1 if interleaved else 0, kv._ref,
                                 batch._struct(T), op, _stream(kv.device)))
    return q_out


def attention(q, kv: PagedKV, batch: PagedBatch, *, scale: float | None = None, out=None):
    """Causal attention of the batch's new tokens over the cache (their own
    keys appended before), every group's prefix included.  q bf16 [T, H, D],
    token stride free; scale: D ** -0.5 by default.  Returns out bf16
    [T, H, D]; padding tokens and tokens that see no key give zero rows."""
    _same_device(kv, batch)
    qp, qs = _heads(q, "q", kv)
    T, H, D = q.shape
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=kv.device)
        op = out.data_ptr()
    else:
        op = _dense(out, torch.bfloat16, "out", q.shape, kv.device)
    b = batch._struct(T)
    nws = lib.bitdelta_attention_workspace(H, kv._ref, b)
    ws = torch.empty((nws,), dtype=torch.uint8, device=kv.device) if nws else None
    check(lib.bitdelta_attention(qp, qs, H, D ** -0.5 if scale is None else scale, kv._ref, b, op,
                                 ws.data_ptr() if nws else 0, nws, _stream(kv.device)))
    return out
