"""GPU tier: the draw of tokens token by token, over rows whose order is known: the
last of the first k for every k, and the token at every place of the running sum."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bd():
    import tenant_fine_tune_amd as bd

    return bd


def every_place(bd, logits, t, rows):
    """Each of the row's tokens is drawn where the definition has it: as the last that
    top-k keeps, and by the random number halfway through its weight.  `rows` at a time."""
    n = logits.shape[0]
    top, order = torch.sort(logits.double(), descending=True, stable=True)
    c = torch.cumsum(torch.exp((top - top[0]) / t), 0)
    before = torch.cat([torch.zeros(1, dtype=torch.float64), c[:-1]])
    # weights differ by 1/32 at most here, so half of one is more than 1 / (3 n) of the whole, far above u's rounding and the sums'
    u = ((before + c) / 2 / c[-1]).float()
    on, k = logits.to(DEV), torch.arange(1, n + 1, dtype=torch.int32, device=DEV)
    for a in range(0, n, rows):
        at = slice(a, min(a + rows, n))
        l = on.expand(at.stop - a, n).contiguous()
        last, _ = bd.sample(l, torch.ones(at.stop - a, device=DEV), temperature=t, top_k=k[at])
        wrong = int((last.cpu().long() != order[at]).sum())
        assert wrong == 0, f"top-k from {a + 1} on: {wrong} wrong"
        drawn, _ = bd.sample(l, u[at].to(DEV), temperature=t)
        wrong = int((drawn.cpu().long() != order[at]).sum())
        assert wrong == 0, f"running sum from place {a} on: {wrong} wrong"


@pytest.mark.parametrize("rows", [200, 1000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("border", [-0.5, -1.0, -2.0, -4.0, 0.5, 1.0, 2.0, 4.0])
def test_neighbours_of_powers_of_two(bd, border, dtype, rows):
    """All bf16 numbers of one bin from a power of two on, many tokens of each, their indexes mixed."""
    step = 2.0 ** -8 * abs(border) * (0.5 if border < 0 else 1.0) * 2
    levels = border + step * torch.arange(0, max(1, int(1 / 32 / step)))
    assert torch.equal(levels.bfloat16().float(), levels)
    g = torch.Generator().manual_seed(3)
    every_place(bd, levels[torch.randint(0, len(levels), (1000,), generator=g)].to(dtype), 1.0, rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("border", [-1.0, -2.0, -4.0, 2.0])
def test_the_last_kept_token_of_a_full_bin(bd, border, dtype):
    """131071 logits of spread 2 as bf16 numbers: every top-k that ends in the bin from a power of two on."""
    n = 131071
    l = (torch.randn(n, generator=torch.Generator().manual_seed(4)) * 2).bfloat16().to(dtype)
    top, order = torch.sort(l.double(), descending=True, stable=True)
    k = (((top >= border) & (top < border + 1 / 32)).nonzero()[:, 0] + 1)
    assert len(k) > 128
    on = l.to(DEV)
    for a in range(0, len(k), 200):
        at = k[a:a + 200]
        rows = on.expand(len(at), n).contiguous()
        last, _ = bd.sample(rows, torch.ones(len(at), device=DEV), top_k=at.int().to(DEV))
        assert int((last.cpu().long() != order[at - 1]).sum()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,size", [(64.0, 2.0 ** -140), (100.0, 2.0 ** -146), (1e10, 1e-38), (1e20, 1e-25), (3e38, 1e-9), (3e38, 1e-20)])
@pytest.mark.parametrize("n", [60, 1000, 6000])
def test_logits_next_to_zero_at_high_temperatures(bd, n, t, size, dtype):
    """Negative logits that scale to nothing share a bin with zero; all weigh the same, so every border is at a whole number."""
    g = torch.Generator().manual_seed(5)
    l = ((torch.rand(n, generator=g, dtype=torch.float64) * 2 - 1.5) * size).to(dtype)
    l[torch.randperm(n, generator=g)[:n // 5]] = 0.0
    l[torch.randperm(n, generator=g)[:n // 9]] = -0.0
    every_place(bd, l, t, 1000)
    # beside logits of ordinary size: only some of the candidates are next to zero
    l[::3] = torch.randn(len(l[::3]), generator=g).to(dtype)
    every_place(bd, l, t, 1000)


@pytest.mark.parametrize("rows", [200, 1000])
def test_ranges_that_meet_at_zero(bd, rows):
    """All tokens alike and too many for one list: smaller ranges of logits, one of which ends right below zero
    (they are cut from the largest logit down, by 2^21 numbers)."""
    g = torch.Generator().manual_seed(6)
    n = 7000
    l = torch.cat([torch.zeros(1500), -torch.zeros(1500), (torch.randperm(2 ** 20, generator=g)[:n - 3001] + 1) * -(2.0 ** -149),
                   torch.tensor([1.25 - 2.0 ** -23])])[torch.randperm(n, generator=g)]
    assert int(l.max().view(torch.int32)) & 0x1FFFFF == 0x1FFFFF and len(l.unique()) == n - 3001 + 2
    every_place(bd, l, float("inf"), rows)
