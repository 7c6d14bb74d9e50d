"""GPU tier: attention over values that are not finite, in tiles that every row
sees whole and in tiles that some rows see in part."""
import numpy as np
import pytest
import torch

from tests.test_gpu_decoder_ops import NAN, Case, f64

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,ctx", [([2], [70]), ([70], [90]), ([200], [190])])
def test_infinite_values_are_infinite_wherever_the_key_falls(bd, new, ctx, D):
    """w * inf is inf with its sign, inf - inf and NaN are NaN, for a key in the first tile, one in the middle and the
    last token's own, on its own and two in one column."""
    last = ctx[0] + new[0] - 1
    for keys, bad, want in (([0], [INF], INF), ([last], [INF], INF), ([last], [-INF], -INF), ([last - 1], [-INF], -INF),
                            ([last], [NAN], NAN), ([last - 1, last], [INF, INF], INF), ([last - 1, last], [INF, -INF], NAN),
                            ([3, last], [-INF, -INF], -INF), ([3, last], [-INF, INF], NAN), ([last - 1, last], [NAN, INF], NAN)):
        c = Case(new, ctx, 4, 1, D, 16, seed=43)
        plain = bd.attention(c.q, c.kv(bd), c.batch(bd)).clone()
        for j, b in zip(keys, bad):
            c.v[int(c.host.table[0, j // 16]), 0, j % 16, 21] = b
        got = bd.attention(c.q, c.kv(bd), c.batch(bd))
        rest = [i for i in range(D) if i != 21]
        assert torch.equal(got[:, :, rest], plain[:, :, rest]), (keys, bad)
        for t in range(new[0]):
            seen = [b for j, b in zip(keys, bad) if j <= ctx[0] + t]
            col = got[t, :, 21]
            if not seen:
                assert torch.equal(col, plain[t, :, 21]), (keys, bad, t)
            else:
                s = sum(seen)
                assert (col.isnan() if np.isnan(s) else col == s).all(), (keys, bad, t, f64(col))
        assert np.isnan(want) == bool(col.isnan().all())


@pytest.mark.parametrize("new,ctx", [([1], [0]), ([1], [40]), ([70], [9]), ([200], [300])])
def test_rows_whose_scores_are_all_minus_infinity(bd, new, ctx):
    """Keys of -inf against a positive query: such a row is zero, and a row that sees one finite score has its value."""
    c = Case(new, ctx, 2, 1, 64, 16, seed=44)
    c.q[:, :, 0] = 1.0
    c.k[:, 0, :, 0] = -INF
    assert not bd.attention(c.q, c.kv(bd), c.batch(bd)).any()
    last = ctx[0] + new[0] - 1                              # the last token's own key, seen by no other
    pg, sl = int(c.host.table[0, last // 16]), last % 16
    c.k[pg, 0, sl, 0] = 1.0
    out = bd.attention(c.q, c.kv(bd), c.batch(bd))
    assert not out[:-1].any() and torch.equal(out[-1], c.v[pg, :, sl].expand(2, 64))
