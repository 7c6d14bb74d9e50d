"""GPU tier: attention over an 8-bit cache whose scales are zero or negative."""
import pytest
import torch

from tests.test_gpu_decoder_ops import NAN, Case

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


# single tokens, a prompt, a split one, both behind prefixes
BATCHES = [([1, 2], [45, 7], ()), ([70, 3], [9, 40], ()), ([200, 1], [1500, 40], ()), ([1] * 4, [5, 0, 33, 64], [(0, 4, 100)])]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,ctx,groups", BATCHES)
def test_scales_of_any_sign(bd, new, ctx, groups, D):
    """A key scale of zero (a head that held nothing but zeros) makes every score zero and the output the mean of the
    values seen; a negative one turns the order of the scores round."""
    c = Case(new, ctx, 6, 3, D, 16, "e4m3", groups=groups, pad=1, seed=41)
    c.k_scale[0], c.k_scale[1], c.v_scale[2] = 0.0, -c.k_scale[1], -c.v_scale[2]
    out = c.check(bd)
    assert out.isfinite().all()


def test_scale_zero_keeps_what_is_not_finite(bd):
    """0 * NaN and 0 * inf are NaN, in a key or in a query."""
    c = Case([2], [20], 2, 1, 64, 16, "e4m3", seed=42)
    c.k_scale[0] = 0.0
    c.q[0, 0, 3], c.q[1, 1, 3] = NAN, INF
    out = bd.attention(c.q, c.kv(bd), c.batch(bd))
    assert out[0, 0].isnan().all() and out[1, 1].isnan().all()
    assert out[0, 1].isfinite().all() and out[1, 0].isfinite().all()
    c.q[0, 0, 3] = c.q[1, 1, 3] = 0.0
    c.k.view(torch.uint8)[int(c.host.table[0, 0]), 0, 3, 5] = 0x7F
    assert bd.attention(c.q, c.kv(bd), c.batch(bd)).isnan().all()
