"""The 64-bit form of attention over a paged cache, a sequence at a time, for
batches that are too large to go through token by token: the formula and the
bounds of tests/decoder_ref.py."""
from __future__ import annotations

import numpy as np
import torch

from tests.decoder_ref import BF, F32


def sequence_cells(host, s):
    """Of sequence s: its tokens [a, b), the keys that it may see as cells (page, slot), prefix first, and the first
    token of it that sees each (its place among the own keys; none for the prefix)."""
    a, b = int(host.q_start[s]), int(host.q_start[s + 1])
    own = min(max(int(host.kv_len[s]), 0), host.table.shape[1] * host.page)
    g = host.group(s)
    p = 0 if g < 0 else min(max(int(host.prefix_len[g]), 0), host.ptable.shape[1] * host.page)
    pages, slots, first = [], [], []
    for row, n, is_own in ((host.ptable[g] if p else None, p, False), (host.table[s], own, True)):
        if n:
            j = np.arange(n)
            pages.append(row[j // host.page])
            slots.append(j % host.page)
            first.append(j - (own - (b - a)) if is_own else np.full(n, -1 << 40))
    if not pages:
        return a, b, np.zeros(0, int), np.zeros(0, int), np.zeros(0, int)
    pages, slots, first = (np.concatenate(x) for x in (pages, slots, first))
    held = (pages >= 0) & (pages < host.n_pages)
    return a, b, pages[held], slots[held], first[held]


def attention(q, k, v, host, scale):
    """q [T, H, D], k and v [n_pages, H_kv, page, D] (scales applied), starts that do not decrease -> (out, bound)."""
    T, H, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    out, tol = np.zeros((T, H, D)), np.zeros((T, H, D))
    for s in range(len(host.kv_len)):
        a, b, pages, slots, first = sequence_cells(host, s)
        if a == b or not len(pages):
            continue
        kk, vv = (torch.from_numpy(np.ascontiguousarray(x[pages, :, slots].transpose(1, 0, 2))) for x in (k, v))   # [Hk, n, D]
        qq = torch.from_numpy(np.ascontiguousarray(q[a:b].transpose(1, 0, 2).reshape(Hk, G * (b - a), D)))
        seen = torch.from_numpy(np.tile(first[None] <= np.arange(b - a)[:, None], (G, 1)))                           # rows by keys
        z = (qq @ kk.transpose(1, 2).contiguous() * scale).masked_fill(~seen, -np.inf)
        any_seen = seen.any(1)
        top = torch.where(any_seen[:, None], z.amax(2, keepdim=True), torch.zeros(()).double())
        w = torch.exp(z - top)
        w = w / w.sum(2, keepdim=True).clamp(min=1e-300)
        o, mag = w @ vv, w @ vv.abs()
        reach = (qq.abs() @ kk.abs().transpose(1, 2).contiguous()).masked_fill(~seen, 0.0).amax(2, keepdim=True)
        dz = 2 * (D + 8) * F32 * scale * reach
        t = BF * o.abs() + (BF + dz + 2.0 ** -18) * mag * (1 + BF)
        for dst, src in ((out, o), (tol, t)):
            dst[a:b] = src.numpy().reshape(H, b - a, D).transpose(1, 0, 2)
    return out, tol
