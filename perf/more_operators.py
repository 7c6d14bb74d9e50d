"""From the hidden state to the next token with an 8-bit base, as measured work.

Three operators carry a mixed batch of tenants through linears whose shared
base is held in 8 bits, and from the logits to the drawn token:

  quantize   every token's row x (or a weight's row) as int8 numbers and one scale,
             s = max |x| / 127, q = x / s to the nearest whole number, ties to even
  linear     y[i, r] = s_i (c_r sum_k q[i,k] w[r,k] + alpha_v[r] sum_k q[i,k] sign_v[r,k]): an int8
             base with a scale c per output channel, and the 1-bit delta of token i's variant v
  sample     one token per row of logits: temperature, top-k, top-p, min-p, drawn by a given
             random number

`run` computes them in plain torch (own = False) or through the package
(own = True); `exact` is the definition in 64 bits.  Matrix shapes of the larger
cases are those of the 70B-class stack; vocabularies are of usual sizes.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
VARIANTS = 14
_T = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases


def _quantize(name, **kw):
    c = {"name": name, "op": "quantize", "rows": 1, "width": 8192, "dtype": "bf16", "stride_pad": 0}
    c.update(kw)
    return c


def _linear(name, **kw):
    # variants 0: no delta; 1: one delta for every token; above: variant_ids
    c = {"name": name, "op": "linear", "m": 1, "d_out": 8192, "d_in": 8192, "variants": 1, "alpha": "row",
         "out": "bf16", "mix": 1}
    c.update(kw)
    return c


def _sample(name, **kw):
    # style: "open" temperature alone, "nucleus" one setting for all rows, "mixed" each row its own settings
    c = {"name": name, "op": "sample", "rows": 1, "vocab": 32000, "dtype": "bf16", "style": "mixed", "stride_pad": 0,
         "mix": 1}
    c.update(kw)
    return c


def listed():
    return [
        # four tenants' tokens before a linear of a decode step: launch latency
        _quantize("quantize_decode", rows=4),
        # prompts of odd total length before the widest linear of the stack
        _quantize("quantize_prompt", rows=2049, width=28672),
        # one user's next token through one linear of the stack
        _linear("linear_one"),
        # a decode step of 16 tokens of 14 variants through a fused q/k/v projection
        _linear("linear_mixed", m=16, d_out=10240, variants=VARIANTS, mix=2),
        # a larger decode step of an odd number of tokens through the longest rows
        _linear("linear_many", m=61, d_in=28672, variants=VARIANTS, mix=3),
        # logits of 32 tokens over an output head of odd height, kept in fp32 for the draw
        _linear("linear_head", m=32, d_out=50257, variants=0, out="f32", mix=4),
        # a prompt of one variant
        _linear("linear_prompt", m=2048, mix=5),
        # prompts of 14 variants in one batch, some with few tokens
        _linear("linear_prompt_mixed", m=4096, variants=VARIANTS, mix=6),
        # small ragged matrix, one alpha for the matrix of each variant
        _linear("linear_ragged", m=333, d_out=1000, d_in=4104, variants=3, alpha="matrix", out="f32", mix=7),
        # one user's next token, nucleus sampling
        _sample("sample_one", style="nucleus"),
        # a decode step of 64 users, each with settings of their own
        _sample("sample_batch", rows=64, vocab=50257, dtype="f32", mix=2),
        # many answers at once over a large vocabulary of odd size
        _sample("sample_large", rows=512, vocab=131071, mix=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    kind = rng.choice(["quantize", "decode", "decode", "prompt", "prompt", "sample", "sample", "sample"])
    if kind == "quantize":
        width = _log(rng, 64, 32768)
        if rng.random() < 0.75:
            width = max(64, width // 8 * 8)
        c = _quantize("", rows=max(1, min(_log(rng, 1, 16384), 58_000_000 // width)), width=width,
                      dtype=rng.choice(["bf16", "bf16", "f32"]), stride_pad=rng.choice([0, 0, 8, 24]))
    elif kind == "sample":
        vocab = _log(rng, 2, 262144)
        rows = max(1, min(_log(rng, 1, 1024), 67_000_000 // vocab))
        c = _sample("", rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
                    style=rng.choice(["open", "nucleus", "mixed", "mixed"]), stride_pad=rng.choice([0, 0, 1, 24]),
                    mix=rng.randrange(1 << 20))
    else:
        decode = kind == "decode"
        d_in = _log(rng, 64, 28672)
        step = rng.choice([8, 64, 64, 256])
        d_in = max(64, d_in // step * step)
        d_out = min(_log(rng, 16, 28672), 235_000_000 // d_in)
        if rng.random() < 0.7:
            d_out = max(16, d_out // 32 * 32)
        m = _log(rng, 1, 64) if decode else _log(rng, 65, 4096)
        m = max(1, min(m, int(2.7e11 / (d_in * d_out))))
        c = _linear("", m=m, d_out=d_out, d_in=d_in, variants=rng.choice([0, 1, 1, 3, VARIANTS, VARIANTS]),
                    alpha=rng.choice(["row", "row", "matrix"]), out=rng.choice(["bf16", "bf16", "f32"]),
                    mix=rng.randrange(1 << 20))
    del c["name"]
    return c


def _ids(case):
    """Variant of each token: uneven shares, as tenants have them, in random order."""
    v, m = case["variants"], case["m"]
    rng = random.Random(case["mix"])
    share = [1.0 / (i + 1) ** 1.1 for i in range(v)]
    return rng.choices(range(v), share, k=m)


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["width"]
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + 4 * case["rows"], "flops": n * 4}
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 28 * case["rows"], "flops": n * 8}
    m, n, k = case["m"], case["d_out"], case["d_in"]
    deltas = len(set(_ids(case))) if case["variants"] > 1 else case["variants"]
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": m * k + n * k + deltas * (n * k // 8 + 4 * n) + m * n * out + 4 * n + 8 * m,
            "flops": 2 * m * n * k * (2 if deltas else 1)}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _padded(rows, width, pad, dtype, g, std):
    full = torch.empty(rows, width + pad, dtype=torch.float32, device=DEV).normal_(0, std, generator=g).to(dtype)
    return full[:, :width]


def _quantize_inputs(case, seed):
    g = _gen(seed)
    x = _padded(case["rows"], case["width"], case["stride_pad"], _T[case["dtype"]], g, 1.0)
    # a few columns of activations are far larger than the rest
    cols = torch.randint(0, case["width"], (max(1, case["width"] // 1000),), generator=g, device=DEV)
    x[:, cols] = (x[:, cols].float() * 12.0).to(x.dtype)
    return {"x": x}


def _eight_bits(rows, width, std, g):
    """Seeded int8 rows and their scales, a slab of rows at a time."""
    q = torch.empty(rows, width, dtype=torch.int8, device=DEV)
    s = torch.empty(rows, dtype=torch.float32, device=DEV)
    slab = max(1, (1 << 26) // width)
    for a in range(0, rows, slab):
        x = torch.empty(min(slab, rows - a), width, device=DEV).normal_(0, std, generator=g)
        s[a:a + slab] = x.abs().amax(1) / 127.0
        q[a:a + slab] = (x / s[a:a + slab, None]).round_().clamp_(-127, 127).to(torch.int8)
    return q, s


def _linear_inputs(case, seed):
    g = _gen(seed)
    m, n, k, v = case["m"], case["d_out"], case["d_in"], case["variants"]
    s = {}
    s["q"], s["q_scale"] = _eight_bits(m, k, 1.0, g)
    s["w"], s["w_scale"] = _eight_bits(n, k, 0.02, g)
    s["signs"] = s["alpha"] = s["ids"] = None
    if v:
        lead = (v,) if v > 1 else ()
        s["signs"] = torch.randint(0, 256, (*lead, n, k // 8), generator=g, device=DEV, dtype=torch.uint8)
        shape = (*lead, n) if case["alpha"] == "row" else (v,)
        s["alpha"] = torch.empty(shape, device=DEV).normal_(0, 0.5, generator=g).exp_().mul_(1e-3)
    if v > 1:
        ids = _ids(case)
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
        s["rows"] = {i: torch.tensor([t for t, w in enumerate(ids) if w == i], device=DEV) for i in sorted(set(ids))}
    elif v:
        s["rows"] = {0: torch.arange(m, device=DEV)}
    return s


def _sample_inputs(case, seed):
    g = _gen(seed)
    rng = random.Random(seed * 7919 + case["mix"])
    m, v = case["rows"], case["vocab"]
    logits = _padded(m, v, case["stride_pad"], torch.float32, g, 2.0)
    # a few tokens of a row stand out by far
    n = min(v, 40)
    at = torch.randint(0, v, (m, n), generator=g, device=DEV)
    lift = torch.empty(m, n, device=DEV).exponential_(0.4, generator=g)
    logits.scatter_add_(1, at, lift + 3.0)
    s = {"logits": logits if case["dtype"] == "f32" else logits.to(torch.bfloat16)}
    s["u"] = torch.rand(m, generator=g, device=DEV)
    f32 = dict(dtype=torch.float32, device=DEV)
    if case["style"] == "open":
        s["temperature"] = torch.tensor([rng.choice([0.7, 1.0, 1.2]) for _ in range(m)], **f32)
        s["top_k"] = s["top_p"] = s["min_p"] = None
    elif case["style"] == "nucleus":
        s["temperature"], s["top_p"] = torch.full((m,), 0.7, **f32), torch.full((m,), 0.9, **f32)
        s["top_k"] = s["min_p"] = None
    else:
        s["temperature"] = torch.tensor([rng.choice([0.0, 0.3, 0.7, 0.8, 1.0, 1.0, 1.3]) for _ in range(m)], **f32)
        s["top_k"] = torch.tensor([rng.choice([0, 0, 1, 20, 50, 1000, rng.randint(1, v)]) for _ in range(m)],
                                  dtype=torch.int32, device=DEV)
        s["top_p"] = torch.tensor([rng.choice([1.0, 1.0, 0.5, 0.9, 0.95]) for _ in range(m)], **f32)
        s["min_p"] = torch.tensor([rng.choice([0.0, 0.0, 0.02, 0.1]) for _ in range(m)], **f32)
    return s


_INPUTS = {"quantize": _quantize_inputs, "linear": _linear_inputs, "sample": _sample_inputs}


def prepare(case, seed):
    s = _INPUTS[case["op"]](case, seed)
    s["case"] = case
    return s


# --------------------------------------------------------------------- run


def run(state):
    return {"quantize": _run_quantize, "linear": _run_linear, "sample": _run_sample}[state["case"]["op"]](state)


def _run_quantize(s):
    if own:
        import tenant_fine_tune_amd as bd

        return bd.quantize_int8(s["x"])
    x = s["x"].double()          # 64 bits: a quotient next to a half must not round on to it
    scale = (x.abs().amax(1) / 127.0).float()
    div = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    q = (x / div[:, None]).round_().clamp_(-127, 127)
    return q.to(torch.int8), scale


def _unpacked(bits):
    """+1 / -1 in 32 bits from packed signs, bit j of byte b being column 8 b + j."""
    shift = torch.arange(8, device=bits.device, dtype=torch.uint8)
    return ((bits[..., None] >> shift) & 1).flatten(-2).float().mul_(2.0).sub_(1.0)


def _run_linear(s):
    c = s["case"]
    if own:
        import tenant_fine_tune_amd as bd

        return bd.linear_int8(s["q"], s["q_scale"], s["w"], s["w_scale"], s["signs"], s["alpha"],
                              variant_ids=s["ids"], per_matrix=c["alpha"] == "matrix", out_dtype=_T[c["out"]])
    x = s["q"].float()
    y = torch.matmul(x, s["w"].float().T) * s["w_scale"]
    if c["variants"]:
        for v, rows in s["rows"].items():
            signs, alpha = (s["signs"][v], s["alpha"][v]) if c["variants"] > 1 else (s["signs"], s["alpha"])
            y[rows] += torch.matmul(x[rows], _unpacked(signs).T) * alpha
    return (y * s["q_scale"][:, None]).to(_T[c["out"]])


def _run_sample(s):
    if own:
        import tenant_fine_tune_amd as bd

        return bd.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                         min_p=s["min_p"])
    # 64 bits: which token is drawn is decided next to a border of the running sum
    top, order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    m, v = top.shape
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    z = (top - top[:, :1].double()) / torch.where(greedy, torch.ones_like(t), t)
    w = torch.exp(z)
    cum = torch.cumsum(w, 1)
    before = cum - w
    rank = torch.arange(v, device=top.device)
    keep = torch.ones(m, v, dtype=torch.bool, device=top.device)
    total = cum[:, -1:]
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        k = torch.where(k <= 0, torch.full_like(k, v), k.clamp(max=v))
        keep &= rank < k
        total = cum.gather(1, k - 1)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        keep &= (before < p * total) | (p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    keep[:, 0] = True
    keep &= (rank == 0) | ~greedy
    n = keep.sum(1, keepdim=True)
    total = cum.gather(1, n - 1)
    at = torch.minimum(((cum <= s["u"].double()[:, None] * total) & keep).sum(1, keepdim=True), n - 1)
    prob = torch.where(greedy, torch.ones_like(total), w.gather(1, at) / total)
    return order.gather(1, at)[:, 0].int(), torch.log(prob)[:, 0].float()


# ------------------------------------------------------------------- exact


def exact(case, seed):
    s = _INPUTS[case["op"]](case, seed)
    if case["op"] == "quantize":
        x = s["x"].double()
        top = torch.maximum(x.max(1).values, -x.min(1).values)
        step = (top / 127).float().double()        # a scale is the 32-bit number that is stored
        ratio = torch.where(step[:, None] > 0, x / step[:, None], torch.zeros_like(x))
        low = torch.floor(ratio)
        up = (ratio - low > 0.5) | ((ratio - low == 0.5) & (torch.remainder(low, 2) == 1))
        return torch.clamp(low + up, -127, 127).to(torch.int8), top / 127
    if case["op"] == "linear":
        w, x = s["w"].double(), s["q"].double()
        y = torch.empty(case["m"], case["d_out"], dtype=torch.float64, device=DEV)
        which = s["ids"].long() if s["ids"] is not None else torch.zeros(case["m"], dtype=torch.long, device=DEV)
        for a in range(0, case["m"], 512):
            y[a:a + 512] = torch.matmul(x[a:a + 512], w.T) * s["w_scale"].double()
        if case["variants"]:
            packed, alpha = s["signs"].view(-1, case["d_out"], case["d_in"] // 8), s["alpha"].double()
            alpha = alpha.view(max(1, case["variants"]), -1)
            for v in range(case["variants"]):
                mine = torch.nonzero(which == v)[:, 0]
                if mine.numel() == 0:
                    continue
                b = torch.stack([(packed[v] // (1 << j)) % 2 for j in range(8)], -1).flatten(1).double()
                z = x[mine]
                y[mine] += (2.0 * torch.matmul(z, b.T) - z.sum(1, keepdim=True)) * alpha[v]
        return y * s["q_scale"].double()[:, None]
    # one row at a time: probabilities in order, then the limits one after another
    tokens, logs = [], []
    v = case["vocab"]
    for i in range(case["rows"]):
        temp = float(s["temperature"][i])
        neg, order = torch.sort(-s["logits"][i].double(), stable=True)
        if temp <= 0:
            tokens.append(order[0])
            logs.append(torch.zeros((), dtype=torch.float64, device=DEV))
            continue
        kept = v
        if s["top_k"] is not None and 0 < int(s["top_k"][i]) < v:
            kept = int(s["top_k"][i])
        prob = torch.softmax(-neg[:kept] / temp, 0)
        upto = torch.cumsum(prob, 0)
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            kept = min(kept, int((upto < float(s["top_p"][i])).sum()) + 1)
        if s["min_p"] is not None:
            kept = min(kept, max(1, int((prob >= float(s["min_p"][i]) * prob[0]).sum())))
        upto = upto[:kept] / upto[kept - 1]
        j = min(int(torch.searchsorted(upto, s["u"][i].double(), right=True)), kept - 1)
        tokens.append(order[j])
        logs.append(torch.log(prob[j] / prob[:kept].sum()))
    return torch.stack(tokens).int(), torch.stack(logs)
