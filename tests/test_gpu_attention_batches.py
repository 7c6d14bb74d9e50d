"""GPU tier: attention over batches of unusual make-up or size: hundreds and
thousands of sequences and tokens, where a call's work is listed, split and
joined in other ways than for a few."""
import numpy as np
import pytest
import torch

from tests import decoder_ref as ref
from tests import decoder_ref_batch as ref_batch
from tests.test_gpu_decoder_ops import DEV, NAN, Case, close, f64, gen, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


def test_padding_alone_with_groups(bd):
    """No sequences, no arrays of sequences, groups that are still there: zero rows."""
    import ctypes

    from tenant_fine_tune_amd import decoder

    kv = bd.PagedKV.empty(4, 2, 16, 64)
    start, lens, table = i32([0, 3]), i32([40]), i32([[0, 1, 2]])
    b = decoder._Batch(None, None, None, start.data_ptr(), lens.data_ptr(), table.data_ptr(), 5, 0, 0, 1, 3, 0)
    q = torch.ones(5, 8, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.ones_like(q)
    need = bd.lib.bitdelta_attention_workspace(8, kv._ref, ctypes.addressof(b))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    assert bd.lib.bitdelta_attention(q.data_ptr(), 512, 8, 0.1, kv._ref, ctypes.addressof(b), out.data_ptr(),
                                     ws.data_ptr(), need, st) == bd.BD_OK
    assert not out.any()
    out.fill_(1)
    k = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert bd.lib.bitdelta_kv_append(q.data_ptr(), 512, k.data_ptr(), 128, k.data_ptr(), 128, 8, None, 0, 0, kv._ref,
                                     ctypes.addressof(b), out.data_ptr(), st) == bd.BD_OK
    assert not out.any()


class Many(Case):
    """A Case whose dead cells are filled, and whose answers are formed, a sequence at a time."""

    def __init__(self, new, ctx, H, Hk, D, page, cache="bf16", **kw):
        super().__init__(new, ctx, H, Hk, D, page, cache, fill=False, **kw)
        live = np.zeros((self.n_pages, page), bool)
        for s in range(len(new)):
            _, _, pages, slots, _ = ref_batch.sequence_cells(self.host, s)
            live[pages, slots] = True
        dead = torch.from_numpy(~live)[:, None, :, None].to(DEV)
        for name in ("k", "v"):
            t = getattr(self, name)
            setattr(self, name, torch.where(dead, NAN, t.float()).to(t.dtype))

    def check(self, bd):
        out = bd.attention(self.q, self.kv(bd), self.batch(bd))
        want, tol = ref_batch.attention(f64(self.q), *self.values(), self.host, self.D ** -0.5)
        close(out, want, tol, "attention")
        return out


def mixture(seed, n, sizes, ctx_max):
    rng = np.random.default_rng(seed)
    return [int(x) for x in rng.choice(sizes, n)], [int(x) for x in rng.integers(0, ctx_max, n)]


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (64, "e4m3"), (128, "bf16"), (128, "e4m3")])
@pytest.mark.parametrize("n,sizes,tokens", [
    (90, [0, 1, 1, 1, 2, 3, 17, 40, 65], range(513, 2049)),        # a token a workgroup in the join
    (170, [0, 1, 1, 2, 5, 16, 17, 30, 55], range(2049, 6000)),    # sixteen: prompts, padding and single tokens in one
])
def test_mixtures_of_many_tokens(bd, n, sizes, tokens, D, cache):
    """Streamed, finished, split and padding tokens side by side, part of them behind shared and own prefixes."""
    new, ctx = mixture(n + D, n, sizes, 300)
    new[3], new[n // 2], new[n - 2] = 150, 201, 0
    assert sum(new) in tokens
    groups = [(0, 1, 70), (1, 30, 33), (30, 40, 0), (40, n // 2 - 1, 130), (n // 2 - 1, n, 64)]
    Many(new, ctx, 4, 2, D, 16, cache, groups=groups, pad=37, seed=n).check(bd)
    Many(new, ctx, 3, 1, D, 32, cache, pad=21, seed=n + 1).check(bd)


@pytest.mark.parametrize("H,D,new,groups", [
    (128, 64, [500, 33, 1, 1, 0, 600, 700, 300], []),
    (128, 64, [1, 1, 700, 40, 2, 760, 600], [(0, 2, 70), (2, 4, 130), (4, 7, 0)]), (64, 128, [3, 600, 1, 1, 500, 1001], []),
])
def test_prompts_that_fill_the_chip_without_splits(bd, H, D, new, groups):
    """So many row tiles that no sequence's keys are split; a shared prefix still leaves states."""
    ctx = [5, 60, 0, 31, 200, 9, 64, 1][:len(new)]
    assert -(-sum(new) // (256 if D == 64 else 128)) * H >= 1024
    Many(new, ctx, H, H, D, 64, groups=groups, pad=3, seed=H).check(bd)


@pytest.mark.parametrize("n,n_groups", [(1000, 0), (257, 3), (700, 200), (4096, 0), (4096, 256)])
def test_many_sequences(bd, n, n_groups):
    """Several sequences a thread where the batch is listed, groups among them."""
    rng = np.random.default_rng(n + n_groups)
    new, ctx = mixture(n, n, [1, 1, 1, 1, 0, 2], 90)
    new[n // 3], new[n - 1] = 50, 20
    groups = []
    if n_groups:
        bounds = [0, *np.sort(rng.choice(np.arange(1, n - 3), n_groups - 1, replace=False)), n - 3]
        groups = [(int(a), int(b), int(rng.integers(0, 100))) for a, b in zip(bounds, bounds[1:])]
    Many(new, ctx, 4, 1, 64, 16, groups=groups, pad=5, seed=n).check(bd)
    # single tokens alone
    Many([1] * n, ctx, 4, 2, 64, 16, seed=n + 1).check(bd)


def test_append_of_many_sequences(bd):
    """Every token's place and position among thousands of sequences and hundreds of groups."""
    n = 3000
    new, ctx = mixture(5, n, [0, 1, 1, 2, 7], 60)
    groups = [(i * 11, (i + 1) * 11, 1 + i * 977 % 3000) for i in range(256)]
    c = Case(new, ctx, 2, 1, 64, 16, pad=9, seed=6, fill=False)
    c.groups = groups
    c.host.group_start, c.host.prefix_len = np.array([a for a, _, _ in groups] + [groups[-1][1]]), [p for _, _, p in groups]
    c.host.ptable = np.zeros((256, 3000 // 16 + 1), np.int32)
    g = gen(8)
    q, k, v = randn(g, c.T, 2, 64).to(DEV), randn(g, c.T, 1, 64).to(DEV), randn(g, c.T, 1, 64).to(DEV)
    inv = torch.tensor([1.0, 0.3, 0.1, 0.03, 0.01, 3e-3, 1e-3, 0.0], dtype=torch.float64)
    got = bd.kv_append(q, k, v, inv.to(DEV), c.kv(bd), c.batch(bd))
    hq, hk, hv, gq, gk, gv = f64(q), f64(k), f64(v), f64(got), f64(c.k), f64(c.v)
    seq = np.repeat(np.arange(n), new)
    assert not gq[len(seq):].any()
    for t, s in enumerate(seq):
        at = ctx[s] + t - int(c.host.q_start[s])
        gi = s // 11 if s < groups[-1][1] else -1
        pos = at + (groups[gi][2] if gi >= 0 else 0)
        pg, sl = c.host.cell(c.host.table[s], at)
        assert np.array_equal(gv[pg, :, sl], hv[t]), (t, s)
        for have, x in ((gq[t], hq[t]), (gk[pg, :, sl], hk[t])):
            y, mag = ref.rotate(x, pos, inv.numpy(), False)
            assert (np.abs(have - y) <= ref.BF * (np.abs(y) + 2.0 ** -20 * mag) + 2.0 ** -20 * mag).all(), (t, s)
