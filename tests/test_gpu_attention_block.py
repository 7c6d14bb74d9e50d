"""GPU tier: the attention half of a decoder layer (block.AttentionBlock) over
a mixed batch of variants: a prompt, then single tokens, behind a shared
prefix, against the same layer in 64 bits with bf16 roundings at the same
places."""
import numpy as np
import pytest
import torch

import synth
from tests import decoder_ref as ref
from tests.gpu_util import bf16_dev, f32_dev, u8_dev

pytestmark = pytest.mark.gpu

V, D, H, HK, DM, PAGE = 3, 64, 4, 2, 256, 16


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


def bf(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double().numpy()


def projection(bd, rows, cols, seed):
    """Base, signs and alpha of V variants, and the variants' effective weights in 64 bits."""
    wb = bf16_dev(synth.to_bf16_bits(synth.normal_f32((rows, cols), cols ** -0.5, seed, 8101)))
    signs = u8_dev(synth.u64((V, rows, cols // 8), seed, 8102).astype(np.uint8))
    alpha = f32_dev(np.abs(synth.normal_f32((V, rows), 0.2 * cols ** -0.5, seed, 8103)) + np.float32(1e-4))
    eff = [bd.reconstruct(wb, signs[v].contiguous(), alpha[v].contiguous(), per_matrix=False) for v in range(V)]
    return (wb, signs, alpha), [e.double().cpu().numpy() for e in eff]


def test_prompt_then_tokens(bd):
    from tenant_fine_tune_amd.block import AttentionBlock

    qkv, wq = projection(bd, (H + 2 * HK) * D, DM, 1)
    out, wo = projection(bd, DM, H * D, 2)
    g = torch.Generator().manual_seed(3)
    post, nxt = ((1 + torch.randn(V, DM, generator=g) * 0.2).to(torch.bfloat16) for _ in range(2))
    inv = torch.tensor(10000.0, dtype=torch.float64) ** (-torch.arange(32, dtype=torch.float64) / 32)
    kv = bd.PagedKV.empty(24, HK, PAGE, D)
    kv.k.fill_(float("nan"))
    kv.v.fill_(float("nan"))
    blk = AttentionBlock(qkv, out, H, kv, inv.cuda(), post_weight=post.cuda(), next_weight=nxt.cuda(), scale=0.5)

    # sequence 0 fills the pages of the prefix (40 keys); then 1 and 2 stand behind it
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    prefix = [7, 3, 11]
    tables = [[5, 9, 2], [8, 0, 4]]
    seq_keys = {"p": [], 0: [], 1: []}

    def host(x, residual, ids, owner):
        """One call in 64 bits; owner[t] = (list of its sequence, position, lists it sees)."""
        fused = np.stack([bf(wq[v] @ x[t]) for t, v in enumerate(ids)])
        q = fused[:, :H * D].reshape(-1, H, D)
        k = fused[:, H * D:(H + HK) * D].reshape(-1, HK, D)
        v = fused[:, (H + HK) * D:].reshape(-1, HK, D)
        o = np.zeros((len(ids), H, D))
        for t, (mine, pos, sees) in enumerate(owner):
            seq_keys[mine].append((bf(ref.rotate(k[t], pos, inv.numpy(), False)[0]), v[t]))
            cells = [c for s in sees for c in seq_keys[s]]
            kk, vv = np.stack([c[0] for c in cells]), np.stack([c[1] for c in cells])
            qt = bf(ref.rotate(q[t], pos, inv.numpy(), False)[0])
            for h in range(H):
                z = kk[:, h // 2] @ qt[h] / np.sqrt(D)
                w = np.exp(z - z.max())
                o[t, h] = w @ vv[:, h // 2] / w.sum()
        y = np.stack([bf(wo[v] @ bf(o[t]).reshape(-1)) for t, v in enumerate(ids)])
        r, xn, _, _ = ref.block_norm(residual, y, post.double().numpy(), None, "none", 0.5, nxt.double().numpy(),
                                     np.asarray(ids), 1e-6)
        return xn, r

    def run(n, ids, batch, owner):
        x = torch.randn(n, DM, generator=g).to(torch.bfloat16)
        res = torch.randn(n, DM, generator=g)
        want_x, want_r = host(x.double().numpy(), res.double().numpy(), ids, owner)
        got_x, got_r = blk.forward(x.cuda(), res.cuda(), i32(ids), batch)
        for got, want in ((got_x, want_x), (got_r, want_r)):
            err = got.double().cpu().numpy() - want
            # five roundings to bf16 on the way, at most 2^-8 each and 2^-9 in the mean: their root sum of squares
            assert np.sqrt((err ** 2).mean()) <= 5 ** 0.5 * 2.0 ** -8 * np.sqrt((want ** 2).mean())

    run(40, [1] * 40, bd.PagedBatch(i32([0, 40]), i32([40]), i32([prefix]), max_new=40),
        [("p", t, ["p"]) for t in range(40)])
    grouped = dict(group_start=i32([0, 2]), prefix_len=i32([40]), prefix_table=i32([prefix]))
    run(23, [1] * 20 + [2] * 3, bd.PagedBatch(i32([0, 20, 23]), i32([20, 3]), i32(tables), **grouped),
        [(0, 40 + t, ["p", 0]) for t in range(20)] + [(1, 40 + t, ["p", 1]) for t in range(3)])
    for step in range(2):
        run(2, [0, 2], bd.PagedBatch(i32([0, 1, 2]), i32([21 + step, 4 + step]), i32(tables), max_new=1, **grouped),
            [(0, 60 + step, ["p", 0]), (1, 43 + step, ["p", 1])])
