"""GPU tier: more tokens than one dimension of a launch takes (2^32 threads):
the norm of 2^26 narrow rows and the append of 2^24 tokens."""
import numpy as np
import pytest
import torch

from tests import decoder_ref as ref
from tests.test_gpu_decoder_ops import DEV, close, f64, gen, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


def test_block_norm_of_many_rows(bd):
    m, d = 2 ** 26 + 5, 8
    res = torch.empty(m, d, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    w = (1 + randn(gen(2), 3, d, std=0.3, dtype=torch.float32)).to(torch.bfloat16).to(DEV)
    ids = torch.arange(m, dtype=torch.int32, device=DEV) % 4                     # 3: no such variant
    _, x = bd.block_norm(res, pre_weight=w, variant_ids=ids)
    for a, b in ((0, m // 2), (m // 2, m)):
        _, part = bd.block_norm(res[a:b], pre_weight=w, variant_ids=ids[a:b])
        assert torch.equal(x[a:b], part), (a, b)
    at = [0, 1, 2 ** 20 - 1, 2 ** 20, 2 ** 25 + 1, m - 2, m - 1]
    _, want, _, tol = ref.block_norm(f64(res[at]), pre=f64(w), ids=f64(ids[at]), eps=np.float32(1e-6))
    close(x[at], want, tol, "x")


def test_kv_append_of_many_tokens(bd):
    T, D, page = 2 ** 24 + 3, 64, 1024
    n_pages = T // page + 1
    rng = torch.Generator(DEV).manual_seed(3)
    q, k, v = (torch.empty(T, 1, D, dtype=torch.bfloat16, device=DEV).normal_(generator=rng) for _ in range(3))
    kv = bd.PagedKV.empty(n_pages, 1, page, D)
    order = torch.randperm(n_pages, generator=gen(4)).to(torch.int32)
    batch = bd.PagedBatch(i32([0, T]), i32([T]), order[None].to(DEV), max_new=T)
    inv = torch.tensor([0.7, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 1e-7, 0.0], dtype=torch.float64)
    out = bd.kv_append(q, k, v, inv.to(DEV), kv, batch)
    stored = kv.v[order.long().to(DEV)].view(-1, 1, D)[:T]
    assert torch.equal(stored.view(torch.int16), v.view(torch.int16))
    at = [0, 1, 2 ** 20 - 1, 2 ** 20, 2 ** 22 + 1, 2 ** 24 - 1, 2 ** 24, T - 1]
    for name, got, src in (("q", out, q), ("k", kv.k[order.long().to(DEV)].view(-1, 1, D)[:T], k)):
        for t in at:
            y, mag = ref.rotate(f64(src[t]), t, inv.numpy(), False)
            close(got[t], y, ref.BF * (np.abs(y) + 2.0 ** -20 * mag) + 2.0 ** -20 * mag, (name, t))
        assert torch.equal(got[:, :, 16:].view(torch.int16), src[:, :, 16:].view(torch.int16))
