"""GPU tier: the draw of tokens against its definition in 64 bits (tests/sample_ref.py)."""
import math

import pytest
import torch

from tests import sample_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def bd():
    import tenant_fine_tune_amd as bd

    return bd


def model_like(rows, vocab, seed, std=2.0):
    """Logits as a model gives them: a broad middle and a few tokens far above it."""
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(rows, vocab, generator=g) * std
    n = min(vocab, 30)
    l.scatter_add_(1, torch.randint(0, vocab, (rows, n), generator=g), torch.rand(rows, n, generator=g) * 8)
    return l


def settings(rows, vocab, seed):
    g = torch.Generator().manual_seed(seed + 1000)

    def pick(*values):
        return torch.tensor(values, dtype=torch.float64)[torch.randint(0, len(values), (rows,), generator=g)].float()

    return dict(u=torch.rand(rows, generator=g), t=pick(0.0, 0.2, 0.7, 1.0, 1.0, 1.5, 4.0),
                k=pick(0, 0, 1, 2, 5, 40, 1000, max(1, vocab // 2)).int(), p=pick(1.0, 1.0, 0.1, 0.5, 0.9, 0.999),
                least=pick(0.0, 0.0, 0.01, 0.2))


def matches(bd, logits, u, t, k, p, least, dtype=torch.float32, strided=False):
    logits = logits.to(dtype)
    on = logits.to(DEV)
    if strided:
        room = torch.full((logits.shape[0], logits.shape[1] + 5), 50.0, dtype=dtype, device=DEV)
        room[:, 3:-2] = on
        on = room[:, 3:-2]
    tokens, logs = bd.sample(on, u.to(DEV), temperature=t.to(DEV), top_k=k.to(DEV), top_p=p.to(DEV), min_p=least.to(DEV))
    assert tokens.dtype == torch.int32 and logs.dtype == torch.float32
    ref.check(tokens, logs, logits.float(), u, t, k, p, least)
    return tokens.cpu(), logs.cpu()


def all_rows(rows, u=None, t=1.0, k=0, p=1.0, least=0.0):
    full = torch.full((rows,), 1.0)
    return dict(u=torch.rand(rows, generator=torch.Generator().manual_seed(9)) if u is None else full * u, t=full * t,
                k=(full * k).int(), p=full * p, least=full * least)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 63, 64, 65, 1000, 8191, 8192, 8193, 32000, 50257, 70001, 131072])
def test_model_like_rows(bd, vocab, dtype):
    rows = 64 if vocab <= 8193 else 24
    matches(bd, model_like(rows, vocab, vocab), **settings(rows, vocab, vocab), dtype=dtype)


@pytest.mark.parametrize("rows,vocab", [(1, 1048576), (2, 300001), (700, 129), (1500, 9001)])
def test_many_rows_and_the_largest_vocabulary(bd, rows, vocab):
    matches(bd, model_like(rows, vocab, 5), **settings(rows, vocab, 5))


@pytest.mark.parametrize("limit", [dict(), dict(k=1), dict(k=3), dict(k=500), dict(k=10 ** 6), dict(p=0.0), dict(p=1e-6),
                                   dict(p=0.3), dict(p=0.95), dict(p=1.5), dict(least=1e-4), dict(least=0.5), dict(least=1.0),
                                   dict(least=2.0), dict(k=50, p=0.9, least=0.05), dict(k=-3, p=NAN, least=NAN)])
@pytest.mark.parametrize("t", [0.05, 1.0, 30.0])
def test_each_limit(bd, limit, t):
    matches(bd, model_like(40, 20011, 1), **{**all_rows(40, t=t), **{n: v for n, v in all_rows(40, t=t, **limit).items() if n != "u"}})


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [5, 100, 4096, 4097, 30000, 100003])
def test_ties(bd, vocab, dtype):
    """Equal logits stand in the order of their indexes, also where they are too many to be put in order."""
    rows = 30
    g = torch.Generator().manual_seed(vocab)
    for levels in (1, 2, 5):
        l = torch.randint(0, levels, (rows, vocab), generator=g).float() - 1.0
        s = settings(rows, vocab, vocab + levels)
        s["t"] = s["t"].clamp(min=0.7)
        matches(bd, l, **s, dtype=dtype)


def test_ties_at_the_limits(bd):
    # equal weights: sums are whole, so the borders fall on them exactly
    l = torch.zeros(8, 1000)
    tokens, logs = matches(bd, l, **all_rows(8, u=0.5))
    assert (tokens == 500).all() and torch.allclose(logs, torch.full((8,), -math.log(1000.0)))
    assert (matches(bd, l, **all_rows(8, u=0.0))[0] == 0).all()
    assert (bd.sample(l.to(DEV), torch.full((8,), 1.0 - 2.0 ** -24, device=DEV))[0] == 999).all()
    assert (bd.sample(l.to(DEV), torch.full((8,), 1.0 - 2.0 ** -24, device=DEV), top_p=0.25)[0] == 249).all()
    assert (bd.sample(l.to(DEV), torch.full((8,), 1.0 - 2.0 ** -24, device=DEV), top_k=10)[0] == 9).all()


@pytest.mark.parametrize("spread", [1e-7, 1e-3, 0.2])
@pytest.mark.parametrize("t", [0.5, 1.0, 100.0, INF])
def test_flat_rows(bd, spread, t):
    """Nearly equal logits: thousands of tokens in one bin, found through smaller ones."""
    g = torch.Generator().manual_seed(7)
    l = 3.0 + torch.rand(16, 60000, generator=g) * spread
    s = settings(16, 60000, 3)
    s["t"] = torch.full((16,), t)
    matches(bd, l, **s)


@pytest.mark.parametrize("t", [1e-30, 1e-3, 1e10, 3e38, INF, 2.0 ** -149])
def test_extreme_temperatures(bd, t):
    matches(bd, model_like(20, 5000, 2), **{**settings(20, 5000, 2), "t": torch.full((20,), t)})


@pytest.mark.parametrize("scale", [1e-38, 1e-10, 1e5, 1e30, 1e38])
def test_extreme_logits(bd, scale):
    for t in (1.0, scale):
        matches(bd, model_like(20, 5000, 4) / 20 * scale, **{**settings(20, 5000, 4), "t": torch.full((20,), t)})


@pytest.mark.parametrize("t", [0.0, NAN, -1.0, -INF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_largest_logit(bd, t, dtype):
    l = model_like(30, 70000, 6)
    l[3, 100] = l[3, 60000] = l[3].max()
    l[4] = 1.0
    l[5, ::2] = -INF
    l[6, 77] = INF
    tokens, logs = matches(bd, l, **all_rows(30, t=t), dtype=dtype)
    assert (logs == 0).all() and tokens[4] == 0 and tokens[6] == 77


@pytest.mark.parametrize("t", [0.0, 0.7, INF])
def test_tokens_that_are_not_drawn(bd, t):
    g = torch.Generator().manual_seed(8)
    l = model_like(14, 9000, 8)
    l[0] = -INF
    l[1] = NAN
    l[2, 1:] = -INF
    l[3, :-1] = NAN
    l[4] = l[4].masked_fill(torch.rand(9000, generator=g) < 0.9, -INF)
    l[5] = l[5].masked_fill(torch.rand(9000, generator=g) < 0.5, NAN)
    l[6, 4000] = INF
    l[7, 10::1000] = INF
    l[8] = INF
    l[9, 5] = torch.finfo(torch.float32).max
    l[10] = torch.finfo(torch.float32).min
    l[11] = -0.0
    l[11, ::3] = 0.0
    l[12, ::2] = torch.finfo(torch.float32).min
    for seed in range(3):
        s = settings(14, 9000, seed)
        s["t"] = torch.full((14,), t)
        tokens, logs = matches(bd, l, **s)
        assert tokens[0] == -1 and tokens[1] == -1 and logs[0] == -INF and tokens[2] == 0 and tokens[3] == 8999


@pytest.mark.parametrize("u", [0.0, -1.0, NAN, 1e-30, 0.99999994, 1.0, 2.0, INF])
def test_borders_of_the_random_number(bd, u):
    s = settings(40, 3000, 12)
    s["u"] = torch.full((40,), u)
    s["t"] = s["t"].clamp(min=0.5)
    matches(bd, model_like(40, 3000, 12), **s)


def test_rows_do_not_depend_on_how_they_are_cut(bd):
    """One row alone is cut into more parts than among many: the bits are the same."""
    l, s = model_like(600, 40000, 20).to(DEV), {n: v.to(DEV) for n, v in settings(600, 40000, 20).items()}
    args = lambda i: dict(temperature=s["t"][i], top_k=s["k"][i], top_p=s["p"][i], min_p=s["least"][i])
    tokens, logs = bd.sample(l, s["u"], **args(slice(None)))
    for a in range(0, 600, 37):
        t1, l1 = bd.sample(l[a:a + 1], s["u"][a:a + 1], **args(slice(a, a + 1)))
        assert t1.item() == tokens[a].item() and l1.item() == logs[a].item()
    again = bd.sample(l, s["u"], **args(slice(None)))
    assert torch.equal(again[0], tokens) and torch.equal(again[1], logs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_numbers_for_all_rows_and_outputs(bd, dtype):
    l = model_like(9, 1001, 30)
    matches(bd, l, **settings(9, 1001, 30), dtype=dtype, strided=True)
    l, u = l.to(dtype).to(DEV), torch.rand(9, device=DEV)
    full = lambda v, t=torch.float32: torch.full((9,), v, dtype=t, device=DEV)
    a = bd.sample(l, u, temperature=0.8, top_k=30, top_p=0.9, min_p=0.01)
    b = bd.sample(l, u, temperature=full(0.8), top_k=full(30, torch.int32), top_p=full(0.9), min_p=full(0.01))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out, logs = full(-7, torch.int32), full(3.0)
    c = bd.sample(l[:7], u[:7], temperature=0.8, top_k=30, top_p=0.9, min_p=0.01, out=out[1:8], logprobs_out=logs[1:8])
    assert torch.equal(out[1:8], a[0][:7]) and torch.equal(logs[1:8], a[1][:7]) and c[0].data_ptr() == out[1:].data_ptr()
    assert out[0] == -7 and out[8] == -7 and logs[0] == 3 and logs[8] == 3
    t, g = bd.sample(l[:0], u[:0])
    assert t.shape == (0,) and g.shape == (0,)


def test_draws_follow_the_probabilities(bd):
    """Evenly spaced random numbers meet each token as often as its probability says, off by one at most."""
    l = model_like(1, 300, 40, std=1.0)
    n = 20000
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    tokens, _ = bd.sample(l.expand(n, 300).contiguous().to(DEV), u.float().to(DEV), temperature=0.9)
    p = torch.softmax(l[0].double() / 0.9, 0)
    assert ((torch.bincount(tokens.cpu().long(), minlength=300) - p * n).abs() <= 1.0 + n * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t", [0.3, 0.7, 1.0, 3.0])
def test_a_token_kept_alone_has_logprob_zero(bd, t, dtype):
    g = torch.Generator().manual_seed(17)
    for vocab in (1, 2, 500, 40000):
        logits = torch.randn(9, vocab, generator=g) * 2
        logits[torch.arange(9), torch.randint(0, vocab, (9,), generator=g)] = 9.3
        logits, u = logits.to(dtype).cuda(), torch.rand(9, generator=g).cuda()
        for limit in (dict(top_k=1), dict(top_p=0.0), dict(top_p=1e-5), dict(min_p=1.0), dict(top_k=1, top_p=0.5, min_p=0.9)):
            tokens, logprobs = bd.sample(logits, u, temperature=t, **limit)
            assert torch.equal(tokens.long(), logits.argmax(1)) and (logprobs == 0).all()


@pytest.mark.parametrize("gap", [1.0, 3.0, 8.0, 14.0, 20.0, 25.0])
def test_logprob_next_to_a_probability_of_one(bd, gap):
    g = torch.Generator().manual_seed(18)
    logits = torch.randn(40, 7, generator=g)
    logits[:, 3] = logits.max(1).values + gap
    tokens, logprobs = bd.sample(logits.cuda(), torch.zeros(40).cuda())
    assert (tokens == 3).all()
    l = logits.double()
    others = torch.exp(l - l[:, 3:4])
    others[:, 3] = 0
    others = others.sum(1)
    want = -torch.log1p(others)
    # the weights are off by 2^-37, the sums by a rounding in 64 bits, the output by half a step of fp32
    bound = others * 2.0 ** -35 + 8 * 2.0 ** -53 + want.abs() * 2.0 ** -24
    assert ((logprobs.cpu().double() - want).abs() <= bound).all()


def test_more_rows_than_the_scratch_holds_at_once(bd):
    m, vocab = 40000, 33
    g = torch.Generator().manual_seed(19)
    logits, u = torch.randn(m, vocab, generator=g), torch.rand(m, generator=g)
    k, t = torch.randint(0, 9, (m,), generator=g).int(), torch.rand(m, generator=g) + 0.1
    assert bd.lib.bitdelta_sample_workspace(m, vocab) <= 2 ** 28 + 2 ** 24
    tokens, logprobs = bd.sample(logits.cuda(), u.cuda(), top_k=k.cuda(), temperature=t.cuda(), top_p=0.95, min_p=0.01)
    for at in (0, 16300, 16380, 32760, m - 20):     # either side of where a slice ends, and both ends
        s = slice(at, at + 20)
        ref.check(tokens[s], logprobs[s], logits[s], u[s], t[s], k[s], torch.full((20,), 0.95), torch.full((20,), 0.01))
    again = bd.sample(logits[20000:30000].cuda(), u[20000:30000].cuda(), top_k=k[20000:30000].cuda(),
                      temperature=t[20000:30000].cuda(), top_p=0.95, min_p=0.01)
    assert torch.equal(again[0], tokens[20000:30000]) and torch.equal(again[1], logprobs[20000:30000])
