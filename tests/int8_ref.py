"""Definitions of the 8-bit linears in 64 bits on the CPU, and seeded inputs.

Rounding: a result is rounded once to fp32 and from there to the output's type,
so it is off by at most half a step of that type (finfo.eps / 2 relative), and a
2^-10th of that where the first rounding lands on a tie of the second; the
64-bit products before it add 2^-50 of the terms.
"""
from __future__ import annotations

import torch


def quantized(x):
    """(q int8, scale fp32) of the rows of x (bf16 or fp32), quotients exact."""
    x = x.double().cpu()
    scale = torch.zeros(x.shape[:-1], dtype=torch.float64) if x.shape[-1] == 0 else x.abs().amax(-1) / 127
    scale = scale.float()
    bad = ~torch.isfinite(scale)
    step = scale.double().masked_fill(bad | (scale == 0), 1.0)
    q = (x / step[..., None]).round().clamp(-127, 127)
    q = q.masked_fill((bad | (scale == 0))[..., None], 0.0)
    return q.to(torch.int8), scale.masked_fill(bad, float("nan"))


def signs_of(bits):
    """+1 / -1 in 64 bits from packed signs (least significant bit first)."""
    b = (bits.cpu().to(torch.int32)[..., None] >> torch.arange(8, dtype=torch.int32)) & 1
    return b.flatten(-2).double() * 2 - 1


def linear(q, q_scale, w, w_scale, signs=None, alpha=None, ids=None):
    """(y, size of its terms) in 64 bits; alpha already [N], [1], [V, N] or [V]."""
    q, w, s, c = q.cpu().double(), w.cpu().double(), q_scale.cpu().double(), w_scale.cpu().double()
    y = q @ w.T * c
    size = y.abs()
    if signs is not None:
        n = w.shape[0]
        stacked = signs.cpu().view(-1, n, signs.shape[-1])
        a = alpha.cpu().double().reshape(stacked.shape[0], -1)
        which = torch.zeros(q.shape[0], dtype=torch.long) if ids is None else ids.cpu().long()
        for v in range(stacked.shape[0]):
            rows = (which == v).nonzero()[:, 0]
            if rows.numel():
                d = q[rows] @ signs_of(stacked[v]).T * a[v]
                y[rows] += d
                size[rows] += d.abs()
        out = (which < 0) | (which >= stacked.shape[0])
        y[out] = 0
        size[out] = 0
    return y * s[:, None], size * s[:, None].abs()


def check(y, ref, size):
    eps = torch.finfo(y.dtype).eps
    got = y.cpu().double()
    assert torch.isfinite(got).all()
    tol = ref.abs() * (eps / 2 * (1 + 2.0 ** -10)) + size * 2.0 ** -50 + 2.0 ** -149
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()} off, by up to {float(over.max()):.3e}"


def random_case(m, n, k, variants, seed, per_matrix=False, extremes=False):
    """q, q_scale, w, w_scale, signs, alpha, ids on the CPU; variants 0: no delta, 1: one for all."""
    g = torch.Generator().manual_seed(seed)
    lo, hi = (-128, 128) if extremes else (-127, 128)
    q = torch.randint(lo, hi, (m, k), generator=g, dtype=torch.int8)
    w = torch.randint(lo, hi, (n, k), generator=g, dtype=torch.int8)
    s, c = (torch.rand(r, generator=g) + 0.1 for r in (m, n))
    if not variants:
        return q, s, w, c, None, None, None
    lead = (variants,) if variants > 1 else ()
    signs = torch.randint(0, 256, (*lead, n, k // 8), generator=g, dtype=torch.uint8)
    alpha = torch.rand((max(1, variants),) if per_matrix else (*lead, n), generator=g) * 3 - 1
    ids = torch.randint(0, variants, (m,), generator=g, dtype=torch.int32) if variants > 1 else None
    return q, s, w, c, signs, alpha, ids
