"""GPU tier: a row of a draw among fewer or more others, which decide how it is cut
and how many threads it gets: the bits are the same."""
import pytest
import torch

from tests.test_gpu_sample import model_like, settings

pytestmark = pytest.mark.gpu
DEV = "cuda"


def same_however_many(l, s):
    import tenant_fine_tune_amd as bd

    rows = l.shape[0]
    l, s = l.to(DEV), {n: v.to(DEV) for n, v in s.items()}

    def drawn(a, b):
        return bd.sample(l[a:b], s["u"][a:b], temperature=s["t"][a:b], top_k=s["k"][a:b], top_p=s["p"][a:b], min_p=s["least"][a:b])

    tokens, logs = drawn(0, rows)
    for step in (1, 60, 256, 257, 300):
        for a in range(0, rows, step) if step > 1 else range(0, rows, 7):
            b = min(a + step, rows)
            t, p = drawn(a, b)
            off = int((t != tokens[a:b]).sum()), int((p != logs[a:b]).sum())
            assert off == (0, 0), f"rows {a} to {b}: {off[0]} tokens, {off[1]} logarithms differ"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [300, 5003, 40000, 131071])
def test_rows_among_fewer_and_more_others(vocab, dtype):
    same_however_many(model_like(600, vocab, 21).to(dtype), settings(600, vocab, 21))


@pytest.mark.parametrize("limit", [dict(), dict(p=1.0 - 2.0 ** -24), dict(k=18000), dict(least=1e-13)])
def test_sums_that_their_rounding_decides(limit):
    """Tokens whose weights are next to nothing beside the sum: at the row's end every rounding of the running sums is seen."""
    g = torch.Generator().manual_seed(22)
    l = torch.cat([torch.rand(600, 15000, generator=g) * -6.0, -18.0 - 13.0 * torch.rand(600, 5000, generator=g)], 1)
    s = settings(600, 20000, 22)
    s["u"], s["t"] = torch.tensor([1.0 - 2.0 ** -24, 1.0, 2.0]).repeat(200), torch.ones(600)
    for n, v in dict(k=0, p=1.0, least=0.0).items():
        s[n] = torch.full_like(s[n], limit.get(n, v))
    same_however_many(l[:, torch.randperm(20000, generator=g)], s)
