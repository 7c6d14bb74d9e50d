"""Plain 64-bit forms of the operators between the linears, token by token,
for the tests: the formulas of include/bitdelta_decoder.h in numpy, with the
bounds that each comparison allows.

Roundings are at most half a step: bf16 2^-8, e4m3 2^-4 (2^-10 of the scale
below its normals), fp32 2^-24, relative to the value."""
from __future__ import annotations

import numpy as np

BF, E4, F32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def block_norm(res, block=None, post=None, gate=None, act="none", scale=1.0, pre=None, ids=None, eps=1e-6, res_half=F32):
    """(r', x, bound of r', bound of x); weights [V, d]."""
    m, d = res.shape
    r, x = res.copy(), np.zeros((m, d))
    tr, tx = np.zeros((m, d)), np.zeros((m, d))
    V = (post if post is not None else pre).shape[0] if post is not None or pre is not None else 1
    for i in range(m):
        v = 0 if ids is None else int(ids[i])
        known = 0 <= v < V
        if block is not None and known:
            y = block[i].copy()
            if post is not None:
                y = y / np.sqrt((y * y).mean() + eps) * post[v]
            if gate is not None:
                g = gate[i]
                y = y * {"none": g, "sigmoid": sigmoid(g), "silu": g * sigmoid(g)}[act]
            y = scale * y
            r[i] = res[i] + y
            # a sum of d squares, a root, a quotient, an exponential and four products in fp32
            tr[i] = 2.0 ** -19 * np.abs(y) + 2 * F32 * (np.abs(res[i]) + np.abs(y))
        if pre is not None and known:
            k = 1.0 / np.sqrt((r[i] * r[i]).mean() + eps)
            x[i] = r[i] * k * pre[v]
            rms_err = np.sqrt((tr[i] ** 2).mean()) * k           # the norm's share of the errors of r'
            tx[i] = (BF + 2.0 ** -19 + rms_err) * np.abs(x[i]) + tr[i] * k * np.abs(pre[v]) * (1 + BF)
    return r, x, tr + res_half * (np.abs(r) + tr), tx


class Batch:
    """Host copies of a batch; place(t) gives a token's sequence, place, and visible cells."""

    def __init__(self, q_start, kv_len, table, page, n_pages, group_start=None, prefix_len=None, ptable=None):
        self.q_start, self.kv_len, self.table = np.asarray(q_start), np.asarray(kv_len), np.asarray(table)
        self.page, self.n_pages = page, n_pages
        self.group_start = None if group_start is None else np.asarray(group_start)
        self.prefix_len, self.ptable = prefix_len, None if ptable is None else np.asarray(ptable)

    def seq(self, t):
        for s in range(len(self.kv_len)):
            if self.q_start[s] <= t < self.q_start[s + 1]:
                return s
        return -1

    def group(self, s):
        if self.group_start is not None:
            for g in range(len(self.prefix_len)):
                if self.group_start[g] <= s < self.group_start[g + 1]:
                    return g
        return -1

    def place(self, t):
        s = self.seq(t)
        if s < 0:
            return None
        own = min(max(int(self.kv_len[s]), 0), self.table.shape[1] * self.page)
        at = own - (int(self.q_start[s + 1]) - t)
        g = self.group(s)
        p = 0 if g < 0 else min(max(int(self.prefix_len[g]), 0), self.ptable.shape[1] * self.page)
        return s, at, g, p

    def cell(self, row, j):
        pg = int(row[j // self.page])
        return (pg, j % self.page) if 0 <= pg < self.n_pages else None

    def visible(self, t):
        """Cells (page, slot) that token t sees."""
        pl = self.place(t)
        if pl is None:
            return []
        s, at, g, p = pl
        cells = [self.cell(self.ptable[g], j) for j in range(p)] if p else []
        cells += [self.cell(self.table[s], j) for j in range(at + 1)]
        return [c for c in cells if c is not None]


def rotate(x, pos, inv_freq, interleaved):
    """x [H, D] at one position, and |a| + |b| of each column's pair."""
    y, mag = x.copy(), np.zeros_like(x)
    h = len(inv_freq)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        turns = pos * (inv_freq[i] / (2 * np.pi))
        ang = (turns - np.rint(turns)) * 2 * np.pi
        c, s = np.cos(ang), np.sin(ang)
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
        mag[:, a] = mag[:, b] = np.abs(x[:, a]) + np.abs(x[:, b])
    return y, mag


def attention(q, k, v, batch, scale):
    """q [T, H, D], k and v [n_pages, H_kv, page, D] (scales applied) ->
    (out, bound)."""
    T, H, D = q.shape
    G = H // k.shape[1]
    out, tol = np.zeros((T, H, D)), np.zeros((T, H, D))
    for t in range(T):
        cells = batch.visible(t)
        if not cells:
            continue
        pg, sl = np.array(cells).T
        for h in range(H):
            kk, vv = k[pg, h // G, sl], v[pg, h // G, sl]
            with np.errstate(invalid="ignore"):
                z = kk @ q[t, h] * scale
                w = np.exp(z - z.max())
                w /= w.sum()
                out[t, h] = w @ vv
                mag = w @ np.abs(vv)
                # D products and their sum, the scale and the exponent's argument in fp32, twice (a weight and the sum)
                dz = 2 * (D + 8) * F32 * scale * (np.abs(kk) @ np.abs(q[t, h])).max()
                # the output's rounding, the weights' rounding to bf16, the scores, fp32 sums of the weights
                tol[t, h] = BF * np.abs(out[t, h]) + (BF + dz + 2.0 ** -18) * mag * (1 + BF)
    return out, tol
