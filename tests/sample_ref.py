"""The draw of tokens by its definition, in 64 bits on the CPU, a row at a time,
and how far a border may be from where it is computed to be.

Weights on the GPU are within 2^-37 of themselves (rounding of 1 - w to 2^-36, half
a unit) plus the fp64 operations' roundings, and tokens below exp(-32) of the first may weigh nothing
(at most vocab * exp(-32) of all together).  A running sum relative to the whole is
so within `slack` = 2^-36 + vocab * exp(-32) of its value, and where a border falls
nearer than that to a sum, either neighbour is right.
"""
from __future__ import annotations

import math

import torch


def draw(logits, u, t=1.0, k=0, p=1.0, least=0.0):
    """The tokens that are right for one row, with their log probabilities (one for
    each set of kept tokens that is right)."""
    l = logits.double().cpu()
    l = torch.where(l.isnan(), torch.full_like(l, -math.inf), l)
    order = torch.sort(l, descending=True, stable=True).indices
    top = l[order]
    if top.numel() == 0 or top[0] == -math.inf:
        return {-1: [-math.inf]}
    if not t > 0:
        return {int(order[0]): [0.0]}
    valid = int((top > -math.inf).sum())
    top, order = top[:valid], order[:valid]
    if top[0] == math.inf:
        w = (top == math.inf).double()
    elif t == math.inf:
        w = torch.ones_like(top)
    else:
        w = torch.exp((top - top[0]) / t)
    c = torch.cumsum(w, 0)
    slack = 2.0 ** -36 + l.numel() * math.exp(-32.0)
    n = [min(k, valid) if k > 0 else valid] * 2      # fewest and most tokens kept
    if p < 1:
        whole = float(c[n[0] - 1])
        before = c - w
        for i, s in ((0, -slack), (1, slack)):
            n[i] = min(n[i], max(1, int((before < max(p, 0.0) * whole + s * whole).sum())))
    if least > 0:
        for i, s in ((0, 1e-14), (1, -1e-14)):
            n[i] = min(n[i], max(1, int((w >= min(least, 1.0) * (1 + s)).sum())))
    uu = 0.0 if not u > 0 else min(u, 1.0)
    right = {}
    for kept in range(n[0], n[1] + 1):
        whole = float(c[kept - 1])
        lo = int((c[:kept] <= uu * whole - slack * whole).sum())
        hi = int((c[:kept] <= uu * whole + slack * whole).sum())
        for j in range(lo, min(hi, kept - 1) + 1):
            if w[j] > 0 or j == 0:
                right.setdefault(int(order[j]), []).append(math.log(float(w[j]) / whole) if w[j] > 0 else -math.inf)
    if u >= 1 and not right:
        last = int((w[:n[1]] > 0).sum()) - 1
        right[int(order[last])] = [math.log(float(w[last] / c[n[1] - 1]))]
    return right


def check(tokens, logprobs, logits, u, t, k, p, least):
    """Every row's token is a right one; its logarithm off by half a step of fp32,
    what the weights' roundings add and, where the kept set is in doubt, nothing:
    each right set has its own value."""
    tokens, logprobs = tokens.cpu(), logprobs.cpu()
    for i in range(logits.shape[0]):
        right = draw(logits[i], float(u[i]), float(t[i]), int(k[i]), float(p[i]), float(least[i]))
        got, lp = int(tokens[i]), float(logprobs[i])
        assert got in right, f"row {i}: token {got}, right are {right} (u={u[i]}, t={t[i]}, k={k[i]}, p={p[i]}, min_p={least[i]})"
        slack = 2.0 ** -35 + logits.shape[1] * math.exp(-32.0)
        assert any(lp == r or abs(lp - r) <= abs(r) * 2.0 ** -24 + slack for r in right[got]), (i, lp, right[got])
