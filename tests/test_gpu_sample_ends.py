"""GPU tier: the draw at the ends of the random number's range, where the last tokens weigh
next to nothing beside the row's sum."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [6, 300])
@pytest.mark.parametrize("u", [1.0, 1.5, float("inf")])
def test_from_one_on_the_last_kept_token_is_drawn(u, rows, dtype):
    """Whatever limits leave of a row whose last tokens lie below a 2^-52nd of its sum."""
    import tenant_fine_tune_amd as bd

    g = torch.Generator().manual_seed(31)
    n = 60000
    l = torch.cat([torch.rand(n - 300, generator=g) * -3.0, torch.linspace(-22.0, -31.0, 300)])[torch.randperm(n, generator=g)].to(dtype)
    top, order = torch.sort(l.double(), descending=True, stable=True)
    w = torch.exp(top - top[0])
    on, uu = l.to(DEV).expand(rows, n).contiguous(), torch.full((rows,), u, device=DEV)
    def least(at):
        """A min_p halfway between the weights of two neighbours, so far from both that no rounding decides."""
        after = w[(top < top[at]).nonzero()[0, 0]]
        value = torch.sqrt(w[at] * after).float().double()
        assert after * (1 + 2.0 ** -30) < value < w[at] * (1 - 2.0 ** -30)
        return float(value)

    # of what top-k leaves, top-p keeps what begins below its share; the border is far from every sum
    share, left = float(torch.tensor(0.9999)), n - 200
    begins = torch.cat([torch.zeros(1, dtype=torch.float64), torch.cumsum(w, 0)])[:left] / w[:left].sum()
    assert float((begins - share).abs().min()) > 2.0 ** -30
    cases = [(dict(), n), (dict(top_k=n - 5), n - 5), (dict(top_k=left, top_p=share), int((begins < share).sum())), (dict(top_k=100), 100)]
    cases += [(dict(min_p=least(at)), int((w >= least(at)).sum())) for at in (50, n - 40)]
    for limits, kept in cases:
        tokens, logs = bd.sample(on, uu, **limits)
        assert (tokens.cpu().long() == order[kept - 1]).all(), (limits, int(tokens[0]), int(order[kept - 1]))
        want = torch.log(w[kept - 1] / w[:kept].sum())
        # the weights' and sums' roundings and half a step of fp32
        assert ((logs.cpu().double() - want).abs() <= want.abs() * 2.0 ** -24 + 2.0 ** -35 + n * 2.0 ** -46).all()
