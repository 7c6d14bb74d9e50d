"""GPU tier: block norms whose weights do not depend on the variant (none, or
one row for all) over tokens of many variants: every token gets its block,
whatever its id, and so does a decoder layer's attention half without norms."""
import numpy as np
import pytest
import torch

from tests import decoder_ref as ref
from tests.test_gpu_attention_block import D, DM, H, HK, PAGE, projection
from tests.test_gpu_decoder_ops import close, f64, i32, norm_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


@pytest.mark.parametrize("residual,gate,act", [("f32", False, "none"), ("bf16", True, "silu")])
def test_ids_without_weights(bd, residual, gate, act):
    res, blk, gt, _, _, _ = norm_inputs(9, 1032, 1, residual, "bf16", gate, 0, seed=5)
    ids = i32([0, 1, 2, 7, -1, 13, 4095, 0, 1])
    r, x = bd.block_norm(res, blk, gate=gt, gate_act=act, scale=0.5, variant_ids=ids)
    wr, _, tr, _ = ref.block_norm(f64(res), f64(blk), None, f64(gt), act, 0.5, None, None, np.float32(1e-6),
                                  ref.F32 if residual == "f32" else ref.BF)
    close(r, wr, tr, "residual")
    assert x is None


@pytest.mark.parametrize("which", ["post", "pre", "both"])
def test_ids_with_one_weight_for_all(bd, which):
    res, blk, _, post, pre, _ = norm_inputs(7, 520, 1, "f32", "bf16", False, 0, seed=6)
    ids = i32([0, 1, 2, 7, -1, 13, 0])
    kw = {} if which == "pre" else dict(post_weight=post[0])
    kw.update({} if which == "post" else dict(pre_weight=pre[0]))
    r, x = bd.block_norm(res, blk, variant_ids=ids, **kw)
    wr, wx, tr, tx = ref.block_norm(f64(res), f64(blk), None if which == "pre" else f64(post), None, "none", 1.0,
                                    None if which == "post" else f64(pre), None, np.float32(1e-6))
    close(r, wr, tr, "residual")
    if which == "post":
        assert x is None
    else:
        close(x, wx, tx, "x")


def test_one_row_of_variants_still_has_ids(bd):
    """[1, d] are the weights of variant 0: another id is no variant of theirs."""
    res, blk, _, post, pre, _ = norm_inputs(3, 64, 1, "f32", "bf16", False, 0, seed=7)
    r, x = bd.block_norm(res, blk, post_weight=post, pre_weight=pre, variant_ids=i32([0, 1, -1]))
    assert torch.equal(r[1:], res[1:]) and not x[1:].any() and not torch.equal(r[0], res[0])


def test_attention_half_without_norms(bd):
    """Both norms left out: every variant's tokens get the layer's output added."""
    from tenant_fine_tune_amd.block import AttentionBlock

    qkv, _ = projection(bd, (H + 2 * HK) * D, DM, 1)
    out, _ = projection(bd, DM, H * D, 2)
    g = torch.Generator().manual_seed(4)
    x, res = torch.randn(6, DM, generator=g).to(torch.bfloat16).cuda(), torch.randn(6, DM, generator=g).cuda()
    ids = i32([0, 1, 2, 2, 1, 0])
    kv = bd.PagedKV.empty(8, HK, PAGE, D)
    batch = bd.PagedBatch(i32([0, 4, 6]), i32([4, 2]), i32([[3], [5]]), max_new=4)
    before = f64(res)
    nxt, r = AttentionBlock(qkv, out, H, kv, None, scale=0.5).forward(x, res, ids, batch)
    assert nxt is None and r is res
    q = bd.linear_grouped(x, ids, *qkv, per_matrix=False)[:, :H * D].unflatten(1, (H, D))
    y = f64(bd.linear_grouped(bd.attention(q, kv, batch).flatten(1), ids, *out, per_matrix=False))
    want, _, tol, _ = ref.block_norm(before, y, scale=0.5)
    close(r, want, tol, "residual")


def test_ids_without_weights_through_the_c_abi(bd):
    """No weight pointer: whatever the ids, every row is updated."""
    res, blk, _, _, _, _ = norm_inputs(5, 72, 1, "bf16", "bf16", False, 0, seed=8)
    want, _ = bd.block_norm(res, blk)
    out, ids = torch.zeros_like(res), i32([0, 7, -1, 3, 2])
    rc = bd.lib.bitdelta_block_norm(res.data_ptr(), 72, bd.BD_BF16, blk.data_ptr(), 72, None, 0, 0, 1.0, None, None, 0,
                                    ids.data_ptr(), 3, 5, 72, 1e-6, out.data_ptr(), 72, None,
                                    torch.cuda.current_stream().cuda_stream)
    assert rc == bd.BD_OK
    assert torch.equal(out, want)
