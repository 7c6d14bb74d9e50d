"""CPU tier: what the operators between the linears refuse, through the C ABI
(bad arguments return before any launch, on pointers that nothing
dereferences) and through the binding."""
import ctypes
import math

import pytest
import torch

FAKE, ODD = 4096, 4098


@pytest.fixture(scope="module")
def bd():
    import tenant_fine_tune_amd as bd

    return bd


@pytest.fixture(scope="module")
def dec(bd):
    from tenant_fine_tune_amd import decoder

    return decoder


def norm(bd, **kw):
    a = dict(residual=FAKE, rs=64, rd=0, block=FAKE, bs=64, gate=FAKE, gs=64, act=1, scale=1.0, post=FAKE, pre=FAKE,
             wd=0, ids=FAKE, nv=3, m=2, d=64, eps=1e-6, out=FAKE * 2, os=64, x=FAKE * 3, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return bd.lib.bitdelta_block_norm(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rd=2), "EINVAL"), (dict(wd=-1), "EINVAL"), (dict(act=3), "EINVAL"), (dict(nv=0), "EINVAL"),
    (dict(eps=-1.0), "EINVAL"), (dict(eps=math.nan), "EINVAL"), (dict(m=-1), "ESHAPE"), (dict(m=2 ** 31), "ESHAPE"),
    (dict(d=0), "ESHAPE"), (dict(d=32769), "ESHAPE"), (dict(block=None), "EINVAL"),
    (dict(block=None, gate=None), "EINVAL"), (dict(pre=None, out=None), "EINVAL"), (dict(residual=None), "EINVAL"),
    (dict(rs=63), "ESHAPE"), (dict(bs=63), "ESHAPE"), (dict(gs=0), "ESHAPE"), (dict(os=-64), "ESHAPE"),
    (dict(out=FAKE, rs=72), "EINVAL"), (dict(x=None), "EINVAL"), (dict(residual=4097), "EALIGN"),
    (dict(residual=ODD, rd=1), "EALIGN"), (dict(post=ODD, wd=1), "EALIGN"), (dict(ids=ODD), "EALIGN"),
    (dict(x=4097), "EALIGN"), (dict(out=4097), "EALIGN"), (dict(block=4097), "EALIGN"), (dict(gate=4097), "EALIGN"),
])
def test_block_norm_refuses(bd, kw, status):
    assert norm(bd, **kw) == getattr(bd, "BD_" + status)
    assert bd.lib.bitdelta_last_error()


def test_block_norm_of_nothing(bd):
    assert norm(bd, m=0, residual=None) == bd.BD_OK


CACHE = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, dtype=0, n_pages=9, n_kv_heads=2, page_size=16, head_dim=128)
BATCH = dict(q_start=FAKE, kv_len=FAKE, page_table=FAKE, group_start=None, prefix_len=None, prefix_table=None, n_tokens=4,
             n_seqs=2, max_pages=3, n_groups=0, max_prefix_pages=0, max_new=0)
BAD_CACHE = [
    (dict(dtype=2), "EINVAL"), (dict(n_pages=0), "ESHAPE"), (dict(n_kv_heads=0), "ESHAPE"),
    (dict(n_kv_heads=1025), "ESHAPE"), (dict(page_size=0), "ESHAPE"), (dict(page_size=24), "ESHAPE"),
    (dict(page_size=2048), "ESHAPE"), (dict(head_dim=96), "ESHAPE"), (dict(head_dim=256), "ESHAPE"),
    (dict(k_scale=FAKE), "EINVAL"), (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(k=ODD), "EALIGN"),
    (dict(dtype=1, v_scale=ODD), "EALIGN"),
]
BAD_BATCH = [
    (dict(n_tokens=-1), "ESHAPE"), (dict(n_tokens=2 ** 31), "ESHAPE"), (dict(n_seqs=-1), "ESHAPE"),
    (dict(n_seqs=4097), "ESHAPE"), (dict(n_groups=-1), "ESHAPE"), (dict(n_groups=257), "ESHAPE"),
    (dict(max_new=-1), "ESHAPE"), (dict(max_pages=0), "ESHAPE"), (dict(q_start=None), "EINVAL"),
    (dict(kv_len=None), "EINVAL"), (dict(page_table=None), "EINVAL"), (dict(kv_len=ODD), "EALIGN"),
    (dict(n_groups=1, max_prefix_pages=0, group_start=FAKE, prefix_len=FAKE, prefix_table=FAKE), "ESHAPE"),
    (dict(n_groups=1, max_prefix_pages=2, group_start=FAKE, prefix_len=FAKE), "EINVAL"),
    (dict(n_groups=1, max_prefix_pages=2, group_start=ODD, prefix_len=FAKE, prefix_table=FAKE), "EALIGN"),
]


def structs(dec, cache=(), batch=()):
    c, b = dec._KvCache(**{**CACHE, **dict(cache)}), dec._Batch(**{**BATCH, **dict(batch)})
    return c, b


def append(bd, dec, cache=(), batch=(), **kw):
    c, b = structs(dec, cache, batch)
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, heads=8, inv=FAKE, rotary=128, inter=0,
             cp=ctypes.addressof(c), bp=ctypes.addressof(b), out=FAKE * 2, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return bd.lib.bitdelta_kv_append(*a.values())


def attend(bd, dec, cache=(), batch=(), **kw):
    c, b = structs(dec, cache, batch)
    a = dict(q=FAKE, qs=1024, heads=8, scale=0.1, cp=ctypes.addressof(c), bp=ctypes.addressof(b), out=FAKE * 2,
             ws=None, nws=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return bd.lib.bitdelta_attention(*a.values())


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_cache_refused(bd, dec, kw, status):
    want = getattr(bd, "BD_" + status)
    assert append(bd, dec, cache=kw) == want and attend(bd, dec, cache=kw) == want
    c, b = structs(dec, kw)
    assert bd.lib.bitdelta_attention_workspace(8, ctypes.addressof(c), ctypes.addressof(b)) == 0


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_batch_refused(bd, dec, kw, status):
    want = getattr(bd, "BD_" + status)
    assert append(bd, dec, batch=kw) == want and attend(bd, dec, batch=kw) == want
    c, b = structs(dec, (), kw)
    assert bd.lib.bitdelta_attention_workspace(8, ctypes.addressof(c), ctypes.addressof(b)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(cp=None), "EINVAL"), (dict(bp=None), "EINVAL"), (dict(inter=2), "EINVAL"), (dict(rotary=8), "ESHAPE"),
    (dict(rotary=144), "ESHAPE"), (dict(rotary=-16), "ESHAPE"), (dict(heads=7), "ESHAPE"), (dict(heads=-2), "ESHAPE"),
    (dict(heads=2048), "ESHAPE"), (dict(heads=0), "EINVAL"), (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"),
    (dict(k=ODD), "EALIGN"), (dict(ks=248), "ESHAPE"), (dict(vs=260), "ESHAPE"), (dict(q=None), "EINVAL"),
    (dict(out=None), "EINVAL"), (dict(q=ODD), "EALIGN"), (dict(out=ODD), "EALIGN"), (dict(qs=1020), "ESHAPE"),
    (dict(q=FAKE * 2, qs=1032), "EINVAL"), (dict(inv=None), "EINVAL"), (dict(inv=4100), "EALIGN"),
])
def test_append_refuses(bd, dec, kw, status):
    assert append(bd, dec, **kw) == getattr(bd, "BD_" + status)


@pytest.mark.parametrize("kw,status", [
    (dict(cp=None), "EINVAL"), (dict(bp=None), "EINVAL"), (dict(heads=0), "ESHAPE"), (dict(heads=9), "ESHAPE"),
    (dict(scale=0.0), "EINVAL"), (dict(scale=-1.0), "EINVAL"), (dict(scale=math.inf), "EINVAL"),
    (dict(scale=math.nan), "EINVAL"), (dict(q=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(q=ODD), "EALIGN"),
    (dict(out=ODD), "EALIGN"), (dict(qs=1016), "ESHAPE"), (dict(qs=1028), "ESHAPE"),
])
def test_attention_refuses(bd, dec, kw, status):
    assert attend(bd, dec, **kw) == getattr(bd, "BD_" + status)


def test_attention_workspace_is_asked_for(bd, dec):
    c, b = structs(dec)
    need = bd.lib.bitdelta_attention_workspace(8, ctypes.addressof(c), ctypes.addressof(b))
    if need:
        assert attend(bd, dec, ws=FAKE, nws=need - 1) == bd.BD_EWORKSPACE
        assert attend(bd, dec, ws=None, nws=need) == bd.BD_EINVAL
        assert attend(bd, dec, ws=4104, nws=need) == bd.BD_EALIGN


def test_no_tokens_is_no_work(bd, dec):
    assert append(bd, dec, batch=dict(n_tokens=0), k=None, q=None) == bd.BD_OK
    assert attend(bd, dec, batch=dict(n_tokens=0), q=None) == bd.BD_OK


def test_binding_refuses_host_tensors_and_wrong_types(bd):
    t = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        bd.block_norm(t(2, 8), pre_weight=t(8))
    with pytest.raises(TypeError):
        bd.block_norm(t(2, 8, dt=torch.float16), pre_weight=t(8))
    with pytest.raises(TypeError):
        bd.PagedKV(t(2, 2, 16, 64, dt=torch.float16), t(2, 2, 16, 64, dt=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        bd.PagedKV(t(2, 2, 16, 64), t(2, 2, 16, 64))
    with pytest.raises(TypeError):
        bd.PagedBatch(t(2, dt=torch.int64), t(1, dt=torch.int64), t(1, 1, dt=torch.int64))
    with pytest.raises(AttributeError):
        bd.no_such_operator
