"""CPU tier: what the linears over an 8-bit base and the draw of tokens refuse,
through the C ABI (bad arguments return before any launch, on pointers that
nothing dereferences) and through the binding, and the edges of their workspace
queries."""
import pytest
import torch

FAKE, ODD = 4096, 4098
MAX_WIDTH, MAX_VOCAB, MAX_ROWS = 131064, 1 << 20, 1 << 17


@pytest.fixture(scope="module")
def bd():
    import tenant_fine_tune_amd as bd

    return bd


def call(entry, args, kw):
    assert set(kw) <= set(args)
    return entry(*{**args, **kw}.values())


def quantize(bd, **kw):
    return call(bd.lib.bitdelta_quantize_int8,
                dict(x=FAKE, xs=64, dt=bd.BD_F32, m=2, d=64, q=FAKE, scale=FAKE, stream=None), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), "EINVAL"), (dict(dt=-1), "EINVAL"), (dict(m=-1), "ESHAPE"), (dict(m=2 ** 31), "ESHAPE"),
    (dict(d=0), "ESHAPE"), (dict(d=MAX_WIDTH + 1, xs=2 ** 20), "ESHAPE"), (dict(x=None), "EINVAL"),
    (dict(q=None), "EINVAL"), (dict(scale=None), "EINVAL"), (dict(xs=63), "ESHAPE"), (dict(xs=-64), "ESHAPE"),
    (dict(x=ODD), "EALIGN"), (dict(x=4097, dt=0), "EALIGN"), (dict(scale=ODD), "EALIGN"),
])
def test_quantize_refuses(bd, kw, status):
    assert quantize(bd, **kw) == getattr(bd, "BD_" + status)
    assert bd.lib.bitdelta_last_error()


def linear(bd, **kw):
    return call(bd.lib.bitdelta_linear_int8,
                dict(q=FAKE, qs=FAKE, m=2, w=FAKE, ws=FAKE, signs=FAKE, alpha=FAKE, mode=bd.BD_ALPHA_ROW, ids=FAKE, nv=3,
                     d_out=32, d_in=64, y=FAKE, dt=bd.BD_F32, work=FAKE, nws=1 << 40, stream=None), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(mode=7), "EINVAL"), (dict(dt=2), "EINVAL"), (dict(signs=None), "EINVAL"),
    (dict(signs=None, alpha=None, ids=None), "EINVAL"), (dict(signs=None, alpha=None, nv=0), "EINVAL"),
    (dict(nv=0), "EINVAL"), (dict(nv=-1), "EINVAL"), (dict(nv=4097), "EINVAL"), (dict(ids=None), "EINVAL"),
    (dict(m=-1), "ESHAPE"), (dict(d_in=0), "ESHAPE"), (dict(d_in=60), "ESHAPE"), (dict(d_out=0), "ESHAPE"),
    (dict(d_in=MAX_WIDTH + 8), "ESHAPE"), (dict(d_out=(1 << 26) + 1, d_in=8), "ESHAPE"),
    (dict(m=1 << 26), "ESHAPE"), (dict(d_out=1 << 25), "ESHAPE"), (dict(m=1 << 24, d_in=8), "ESHAPE"),
    (dict(m=1 << 62), "ESHAPE"), (dict(d_out=1 << 62), "ESHAPE"), (dict(d_in=1 << 62), "ESHAPE"),
    (dict(q=None), "EINVAL"), (dict(qs=None), "EINVAL"), (dict(w=None), "EINVAL"), (dict(ws=None), "EINVAL"),
    (dict(alpha=None), "EINVAL"), (dict(y=None), "EINVAL"), (dict(q=4104), "EALIGN"), (dict(w=4104), "EALIGN"),
    (dict(y=4104), "EALIGN"), (dict(qs=ODD), "EALIGN"), (dict(ws=ODD), "EALIGN"), (dict(alpha=ODD), "EALIGN"),
    (dict(ids=ODD), "EALIGN"),
])
def test_linear_refuses(bd, kw, status):
    assert linear(bd, **kw) == getattr(bd, "BD_" + status)
    assert bd.lib.bitdelta_last_error()


@pytest.mark.parametrize("m", [20, 100, 2000])
def test_linear_workspace_is_asked_for(bd, m):
    need = bd.lib.bitdelta_linear_int8_workspace(m, 3, 4096, 4096)
    assert need > 0
    shape = dict(m=m, d_out=4096, d_in=4096)
    assert linear(bd, nws=need - 1, **shape) == bd.BD_EWORKSPACE
    assert linear(bd, work=None, nws=need, **shape) == bd.BD_EINVAL
    assert linear(bd, work=4104, nws=need, **shape) == bd.BD_EALIGN


def test_linear_workspace_over_its_range(bd):
    ask = bd.lib.bitdelta_linear_int8_workspace
    for bad in ((-1, 0, 8, 8), (1, -1, 8, 8), (1, 4097, 8, 8), (1, 0, 0, 8), (1, 0, 8, 4), (2 ** 40, 0, 8, 8), (0, 0, 8, 8),
                (100, 0, 2 ** 62, 8)):
        assert ask(*bad) == 0
    for m in (1, 16, 17, 64, 65, 128, 129, 1000, 16384):
        for n in (1, 16, 1000, 28672):
            for k in (8, 40, 4096, 28672, MAX_WIDTH):
                if m * k >= 2 ** 31 or n * k >= 2 ** 31 or m * n * 2 >= 2 ** 31:
                    continue
                for v in (0, 1, 14, 4096):
                    # at most 2^28 of sums and 2^28 of copies, and a table of the tokens by variant: a number
                    # a token, three a tile
                    assert 0 <= ask(m, v, n, k) <= (1 << (29 if k % 32 else 28)) + 4 * (m + 3 * (m // 64 + v + 2)) + 32


def draw(bd, **kw):
    return call(bd.lib.bitdelta_sample,
                dict(logits=FAKE, ls=100, dt=bd.BD_F32, m=2, vocab=100, u=FAKE, t=None, ta=1.0, k=None, ka=0, p=None, pa=1.0,
                     least=None, la=0.0, tokens=FAKE, logprobs=FAKE, work=FAKE, nws=1 << 40, stream=None), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), "EINVAL"), (dict(m=-1), "ESHAPE"), (dict(m=MAX_ROWS + 1), "ESHAPE"), (dict(vocab=0), "ESHAPE"),
    (dict(vocab=MAX_VOCAB + 1, ls=MAX_VOCAB + 1), "ESHAPE"), (dict(ls=99), "ESHAPE"), (dict(ls=-100), "ESHAPE"),
    (dict(nws=0), "EWORKSPACE"), (dict(logits=None), "EINVAL"), (dict(u=None), "EINVAL"), (dict(tokens=None), "EINVAL"),
    (dict(work=None), "EINVAL"), (dict(work=4104), "EALIGN"), (dict(logits=ODD), "EALIGN"),
    (dict(logits=4097, dt=0), "EALIGN"), (dict(u=ODD), "EALIGN"), (dict(t=ODD), "EALIGN"), (dict(k=ODD), "EALIGN"),
    (dict(p=ODD), "EALIGN"), (dict(least=ODD), "EALIGN"), (dict(tokens=ODD), "EALIGN"), (dict(logprobs=ODD), "EALIGN"),
])
def test_sample_refuses(bd, kw, status):
    assert draw(bd, **kw) == getattr(bd, "BD_" + status)
    assert bd.lib.bitdelta_last_error()


def test_sample_workspace_over_its_range(bd):
    ask = bd.lib.bitdelta_sample_workspace
    for bad in ((-1, 8), (0, 8), (MAX_ROWS + 1, 8), (1, 0), (1, MAX_VOCAB + 1), (2 ** 62, 8), (8, -2 ** 62)):
        assert ask(*bad) == 0
    for m in (1, 7, 512, MAX_ROWS):
        for vocab in (1, 8192, 50257, MAX_VOCAB):
            need = ask(m, vocab)
            assert 0 < need <= 2 ** 28 + 2 ** 24
            assert draw(bd, m=m, vocab=vocab, ls=vocab, nws=need - 1) == bd.BD_EWORKSPACE


def test_no_rows_is_no_work(bd):
    assert quantize(bd, m=0, x=None, q=None, scale=None) == bd.BD_OK
    assert linear(bd, m=0, q=None, qs=None, y=None, ids=None, nv=1, work=None, nws=0) == bd.BD_OK
    assert draw(bd, m=0, logits=None, u=None, tokens=None, work=None, nws=0) == bd.BD_OK


def test_binding_refuses_host_tensors_and_wrong_types(bd):
    t = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    for bad in (t(2, 8, dt=torch.float16), t(2, 8, dt=torch.int8), None, [1.0]):
        with pytest.raises(TypeError):
            bd.quantize_int8(bad)
        with pytest.raises(TypeError):
            bd.sample(bad, t(2))
    with pytest.raises(ValueError, match="GPU"):
        bd.quantize_int8(t(2, 8))
    with pytest.raises(ValueError, match="GPU"):
        bd.quantize_int8(torch.zeros(()))
    with pytest.raises(ValueError, match="GPU"):
        bd.sample(t(2, 8), t(2))
    with pytest.raises(TypeError):
        bd.linear_int8(t(2, 8), t(2), t(4, 8), t(4))
    with pytest.raises(TypeError):
        bd.linear_int8(None, t(2), t(4, 8), t(4))
    with pytest.raises(ValueError, match="GPU"):
        bd.linear_int8(t(2, 8, dt=torch.int8), t(2), t(4, 8, dt=torch.int8), t(4))
