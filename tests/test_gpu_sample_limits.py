"""GPU tier: limits of the draw where tokens are alike."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bd():
    import tenant_fine_tune_amd as bd

    return bd


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("min_p", [1.0 + 2.0 ** -23, 1.5, 3e38, math.inf])
@pytest.mark.parametrize("t", [0.7, 1.0, 1e20, math.inf])
@pytest.mark.parametrize("top", [2.0, -3.0, 1e30, math.inf])
def test_min_p_above_one_keeps_the_first_token(bd, top, t, min_p, dtype):
    """No weight reaches it, and the first token is always kept: the lowest index of equal largest logits."""
    g = torch.Generator().manual_seed(1)
    l = torch.randn(12, 5000, generator=g) - 9.0
    first = torch.empty(12, dtype=torch.long)
    for i in range(12):
        at = torch.randperm(5000, generator=g)[:1 + 300 * i]
        l[i, at] = top
        first[i] = at.min()
    l = l.to(dtype).to(DEV)
    u = torch.linspace(0.0, 1.0, 12, device=DEV)
    for value in (min_p, torch.full((12,), min_p, device=DEV)):
        for more in (dict(), dict(top_k=7), dict(top_p=0.9)):
            tokens, logprobs = bd.sample(l, u, temperature=t, min_p=value, **more)
            assert torch.equal(tokens.cpu().long(), first) and (logprobs == 0).all()
    # one is a weight that the equal ones reach
    tokens, _ = bd.sample(l, torch.ones(12, device=DEV), temperature=t, min_p=1.0)
    ties = l == l.max(1, keepdim=True).values
    if t < 1e20:
        assert torch.equal(tokens.cpu().long(), 4999 - ties.flip(1).int().argmax(1).cpu())


@pytest.mark.parametrize("k", [4000, 9000, 14000, 30000])
@pytest.mark.parametrize("u", [0.01, 0.2])
def test_distant_borders_of_a_million_logits(bd, k, u):
    """The candidates of the last kept token and of the drawn one, and as many or more tokens between them."""
    from tests import sample_ref

    g = torch.Generator().manual_seed(2)
    l = torch.randn(3, 1048576, generator=g) * 2
    uu, one = torch.full((3,), u) + torch.arange(3) * 0.003, torch.ones(3)
    tokens, logprobs = bd.sample(l.to(DEV), uu.to(DEV), top_k=k, min_p=1e-4)
    sample_ref.check(tokens, logprobs, l, uu, one, (one * k).int(), one, torch.full((3,), 1e-4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [4, 300])
def test_borders_in_front_of_many_zeros(bd, rows, dtype):
    """A border among the tokens right below zero, with most of the row at zero."""
    g = torch.Generator().manual_seed(3)
    n, small = 120000, 300
    l = torch.zeros(n)
    l[::2] = -0.0
    at = torch.randperm(n, generator=g)
    l[at[:small]] = -torch.rand(small, generator=g) / 40 - 2.0 ** -20
    l[at[small:2 * small]] = -1.0
    l[at[-1]] = 2.0
    l = l.to(dtype)
    order = torch.sort(l.double(), descending=True, stable=True).indices
    k = n - 2 * small + torch.linspace(1, small, rows).int()
    tokens, _ = bd.sample(l.to(DEV).expand(rows, n).contiguous(), torch.ones(rows, device=DEV), top_k=k.to(DEV))
    assert int((tokens.cpu().long() != order[k.long() - 1]).sum()) == 0


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("t,zero,below", [(3e38, 1e-10, 3e36), (1.0, 0.0, 0.03)])
def test_min_p_below_logits_next_to_zero(bd, t, zero, below, rows):
    """A border of min_p in the bin below zero, too full for a list, with zeros or logits that scale to nothing in front of it."""
    g = torch.Generator().manual_seed(7)
    n = 6000
    l = torch.cat([-torch.rand(n, generator=g) * zero, -torch.rand(n, generator=g) * 0.99 * below - 0.01 * below, torch.full((n,), -3 * below)])
    l = l[torch.randperm(len(l), generator=g)]
    top, order = torch.sort(l.double(), descending=True, stable=True)
    w = torch.exp((top - top[0]) / float(torch.tensor(t)))
    for at in (n + 100, n + n // 2, 2 * n - 100):
        # halfway between two neighbours or, as 32 bits hold it, a step away: no roundings of 64 bits decide
        least = float(torch.sqrt(w[at - 1] * w[at]).float())
        assert float((w - least).abs().min()) > 2.0 ** -45
        kept = int((w >= least).sum())
        tokens, logs = bd.sample(l.to(DEV).expand(rows, len(l)).contiguous(), torch.ones(rows, device=DEV), temperature=t, min_p=least)
        assert int((tokens.cpu().long() != order[kept - 1]).sum()) == 0
        want = torch.log(w[kept - 1] / w[:kept].sum())
        assert ((logs.cpu().double() - want).abs() <= want.abs() * 2.0 ** -24 + 2.0 ** -35).all()
