"""GPU tier: block norms, the append to the paged cache and attention over it
(include/bitdelta_decoder.h) against their 64-bit forms (tests/decoder_ref.py),
at the lengths, masks, strides and page numbers where they can go wrong."""
import numpy as np
import pytest
import torch

from tests import decoder_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)
    bad &= ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]} (bound {tol[bad][0]})")


# -------------------------------------------------------------------- norms

NORMS = [  # m, d, V, residual, weight, gate, act, pad
    (1, 1, 1, "bf16", "bf16", False, "none", 0), (3, 7, 2, "f32", "f32", True, "silu", 1),
    (2, 64, 3, "bf16", "f32", True, "sigmoid", 0), (5, 511, 3, "bf16", "bf16", True, "none", 0),
    (4, 513, 1, "f32", "bf16", False, "none", 3), (3, 2049, 4, "bf16", "bf16", True, "silu", 7),
    (17, 4096, 14, "bf16", "bf16", False, "none", 8), (2, 8192, 14, "f32", "f32", True, "sigmoid", 0),
    (2, 8199, 2, "bf16", "bf16", True, "none", 0), (2, 16384, 2, "f32", "bf16", False, "none", 0),
    (1, 32768, 1, "bf16", "bf16", True, "silu", 0), (300, 72, 5, "bf16", "f32", True, "sigmoid", 0),
    (1100, 1000, 3, "f32", "bf16", True, "silu", 0),
]


def norm_inputs(m, d, V, residual, weight, gate, pad, seed):
    g = gen(seed)
    T = {"bf16": torch.bfloat16, "f32": torch.float32}
    rows = lambda dt, std: randn(g, m, d + pad, std=std, dtype=dt).to(DEV)[:, :d]  # noqa: E731
    res, blk, gt = rows(T[residual], 3.0), rows(torch.bfloat16, 0.6), rows(torch.bfloat16, 2.0) if gate else None
    post, pre = ((1 + randn(g, V, d, std=0.3, dtype=torch.float32)).to(T[weight]).to(DEV) for _ in range(2))
    ids = torch.randint(-1, V + 1, (m,), generator=g, dtype=torch.int32).to(DEV)     # -1 and V: no such variant
    return res, blk, gt, post, pre, ids


@pytest.mark.parametrize("m,d,V,residual,weight,gate,act,pad", NORMS)
def test_block_norm(bd, m, d, V, residual, weight, gate, act, pad):
    res, blk, gt, post, pre, ids = norm_inputs(m, d, V, residual, weight, gate, pad, seed=d)
    r, x = bd.block_norm(res, blk, post_weight=post, gate=gt, gate_act=act, scale=0.7, pre_weight=pre, variant_ids=ids)
    wr, wx, tr, tx = ref.block_norm(f64(res), f64(blk), f64(post), f64(gt), act, np.float32(0.7), f64(pre), f64(ids),
                                    np.float32(1e-6), ref.F32 if residual == "f32" else ref.BF)
    close(r, wr, tr, "residual")
    close(x, wx, tx, "x")


@pytest.mark.parametrize("what", ["pre", "post", "add", "gate"])
def test_block_norm_parts(bd, what):
    """A first norm without a block, a last update without a next norm, a block without a norm of its own."""
    res, blk, gt, post, pre, _ = norm_inputs(9, 1032, 1, "f32", "bf16", True, 0, seed=5)
    kw = {"pre": dict(pre_weight=pre[0]), "post": dict(block=blk, post_weight=post), "add": dict(block=blk, scale=2.0),
          "gate": dict(block=blk, gate=gt, gate_act="silu", pre_weight=pre)}[what]
    r, x = bd.block_norm(res, eps=0.1, **kw)
    wr, wx, tr, tx = ref.block_norm(f64(res), f64(kw.get("block")), f64(kw.get("post_weight")), f64(kw.get("gate")),
                                    "silu" if what == "gate" else "none", kw.get("scale", 1.0),
                                    f64(pre) if "pre_weight" in kw else None, None, np.float32(0.1))
    close(r, wr, tr, "residual")
    if what == "pre":
        assert r is res
    if "pre_weight" in kw:
        close(x, wx, tx, "x")
    else:
        assert x is None


def test_block_norm_in_place_zero_rows_and_empty(bd):
    res, blk, gt, post, pre, ids = norm_inputs(6, 2056, 3, "bf16", "bf16", True, 8, seed=9)
    res[2] = 0
    blk[2] = 0
    want, wx = bd.block_norm(res, blk, post_weight=post, gate=gt, pre_weight=pre, variant_ids=ids)
    got, x = bd.block_norm(res, blk, post_weight=post, gate=gt, pre_weight=pre, variant_ids=ids, residual_out=res)
    assert got is res and torch.equal(got, want) and torch.equal(x, wx)
    assert not x[2].any() and not got[2].any()
    r, x = bd.block_norm(res[:0], blk[:0], post_weight=post, pre_weight=pre, variant_ids=ids[:0])
    assert r.shape == (0, 2056) and x.shape == (0, 2056)


def test_block_norm_refuses_weights(bd):
    res, blk, _, post, pre, ids = norm_inputs(2, 64, 3, "bf16", "bf16", False, 0, seed=4)
    for w, error in ((1.0, TypeError), (pre.half(), TypeError), (pre[0, 0], ValueError), (pre[:0], ValueError),
                     (pre[:, :-1], ValueError), (pre[None], ValueError)):
        with pytest.raises(error, match="weights must be"):
            bd.block_norm(res, blk, pre_weight=w, variant_ids=ids)
    with pytest.raises(ValueError, match="pre_weight"):
        bd.block_norm(res, blk, pre_weight=pre.t().contiguous().t(), variant_ids=ids)
    with pytest.raises(ValueError, match="post_weight must be"):
        bd.block_norm(res, blk, post_weight=post[:2], pre_weight=pre, variant_ids=ids)
    with pytest.raises(ValueError, match="variant_ids"):
        bd.block_norm(res, blk, pre_weight=pre)


def test_block_norm_rows_do_not_mix(bd):
    """A NaN or an infinity stays in its own row."""
    res, blk, _, post, pre, _ = norm_inputs(8, 4104, 1, "bf16", "bf16", False, 0, seed=3)
    want = bd.block_norm(res, blk, post_weight=post, pre_weight=pre)
    blk[3, 5], res[6, 4000] = NAN, float("inf")
    got = bd.block_norm(res, blk, post_weight=post, pre_weight=pre)
    keep = [i for i in range(8) if i not in (3, 6)]
    for w, g in zip(want, got):
        assert torch.equal(w[keep], g[keep])
    assert got[0][3].isnan().all() and got[1][3].isnan().all() and got[1][6, 4000].isnan()


# -------------------------------------------------------------- paged batches


class Case:
    """Random pages for sequences with `new` tokens after `ctx` own keys, groups (first, end, prefix)."""

    def __init__(self, new, ctx, H, Hk, D, page, cache="bf16", groups=(), pad=0, seed=0, fill=True, max_new=None):
        g, rng = gen(seed), np.random.default_rng(seed)
        self.D, self.H, self.Hk, self.page = D, H, Hk, page
        lens = [c + m for c, m in zip(ctx, new)]
        need = [max(0, -(-n // page)) for n in lens] + [-(-p // page) for _, _, p in groups]
        self.n_pages = sum(need) + 2
        order, at = rng.permutation(self.n_pages), 0
        table = np.full((len(new), max([1] + need[:len(new)])), 1 << 30, dtype=np.int32)
        ptable = np.full((max(1, len(groups)), max([1] + need[len(new):])), -7, dtype=np.int32)
        for i, n in enumerate(need):
            row = table[i] if i < len(new) else ptable[i - len(new)]
            row[:n] = order[at:at + n]
            at += n
        q_start = np.concatenate([[0], np.cumsum(new)])
        self.T = int(q_start[-1]) + pad
        gs = pl = None
        if groups:
            gs, pl = [a for a, _, _ in groups] + [groups[-1][1]], [p for _, _, p in groups]
        self.host = ref.Batch(q_start, lens, table, page, self.n_pages, gs, pl, ptable)
        self.groups, self.max_new = groups, max(new) if max_new is None else max_new
        self.q = randn(g, self.T, H, D).to(DEV)
        shape = (self.n_pages, Hk, page, D)
        k, v = randn(g, *shape, std=1.5, dtype=torch.float32), randn(g, *shape, dtype=torch.float32)
        self.k_scale = self.v_scale = None
        if cache == "e4m3":
            self.k_scale, self.v_scale = torch.rand(Hk, generator=g) * 0.01 + 0.03, torch.rand(Hk, generator=g) * 0.01 + 0.03
            k, v = k / self.k_scale.view(1, -1, 1, 1), v / self.v_scale.view(1, -1, 1, 1)
            self.k_scale, self.v_scale = self.k_scale.to(DEV), self.v_scale.to(DEV)
        if fill:     # what no sequence holds: NaN
            live = np.zeros((self.n_pages, page), bool)
            for t in range(self.T):
                for c in self.host.visible(t)[::-1]:
                    if live[c] and t not in q_start:
                        break
                    live[c] = True
            dead = torch.from_numpy(~live)[:, None, :, None]
            k, v = torch.where(dead, NAN, k), torch.where(dead, NAN, v)
        dt = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
        self.k, self.v = k.to(dt).to(DEV), v.to(dt).to(DEV)

    def batch(self, bd):
        h = self.host
        kw = {} if not self.groups else dict(group_start=i32(h.group_start), prefix_len=i32(h.prefix_len),
                                             prefix_table=i32(h.ptable))
        return bd.PagedBatch(i32(h.q_start), i32(h.kv_len), i32(h.table), max_new=self.max_new, **kw)

    def kv(self, bd):
        return bd.PagedKV(self.k, self.v, k_scale=self.k_scale, v_scale=self.v_scale)

    def values(self):
        s = [1.0 if x is None else f64(x).reshape(1, -1, 1, 1) for x in (self.k_scale, self.v_scale)]
        return f64(self.k) * s[0], f64(self.v) * s[1]

    def check(self, bd, scale=None, q=None):
        q = self.q if q is None else q
        out = bd.attention(q, self.kv(bd), self.batch(bd), scale=scale)
        want, tol = ref.attention(f64(q), *self.values(), self.host, self.D ** -0.5 if scale is None else scale)
        close(out, want, tol, "attention")
        return out


DECODE = [  # new, ctx, H, Hk, D, page
    ([1], [0], 1, 1, 64, 1), ([1], [0], 8, 1, 128, 16), ([1], [30], 16, 2, 128, 8), ([1], [31], 5, 5, 64, 32),
    ([1], [32], 14, 2, 64, 16), ([1], [1000], 64, 8, 128, 16), ([1] * 9, [0, 1, 14, 15, 16, 63, 64, 65, 500], 24, 8, 128, 16),
    ([1, 0, 1, 2, 1], [70, 40, 0, 129, 255], 32, 4, 64, 64), ([1] * 40, list(range(0, 400, 10)), 7, 1, 128, 256),
    ([3, 1, 4], [5, 300, 0], 8, 2, 128, 4), ([1, 1], [5000, 17], 48, 4, 64, 1024), ([2, 2, 2], [90, 0, 7], 16, 16, 128, 2),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,ctx,H,Hk,D,page", DECODE)
def test_attention_decode(bd, new, ctx, H, Hk, D, page, cache):
    Case(new, ctx, H, Hk, D, page, cache, pad=2, seed=len(new) + H).check(bd)


PROMPT = [
    ([33], [0], 8, 1, 128, 16), ([128], [0], 4, 4, 64, 16), ([129, 1, 0, 64], [0, 0, 0, 0], 6, 2, 128, 32),
    ([65, 1, 1, 1], [200, 30, 0, 511], 8, 2, 64, 8), ([17, 300], [1, 63], 5, 1, 128, 64), ([257], [70], 2, 1, 128, 128),
    ([70, 40], [0, 20], 16, 1, 64, 16), ([1] * 20 + [90], [5] * 21, 12, 4, 128, 16),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,ctx,H,Hk,D,page", PROMPT)
def test_attention_prompt(bd, new, ctx, H, Hk, D, page, cache):
    Case(new, ctx, H, Hk, D, page, cache, pad=1, seed=len(new) + H + D).check(bd)


PREFIX = [  # new, ctx, groups
    ([1] * 6, [0, 3, 20, 0, 1, 64], [(0, 3, 100), (3, 6, 31)]), ([1] * 5, [4] * 5, [(0, 5, 1)]),
    ([1, 0, 2, 1], [9, 0, 70, 0], [(0, 4, 333)]), ([1] * 4, [2] * 4, [(1, 3, 70)]), ([1, 1, 1], [5, 6, 7], [(0, 1, 64), (1, 1, 9), (1, 3, 0)]),
    ([40, 7, 1], [0, 9, 2], [(0, 2, 130), (2, 3, 77)]), ([1] * 33, [3] * 33, [(0, 33, 513)]),
]


@pytest.mark.parametrize("H,Hk,D,page,cache", [(8, 1, 128, 16, "bf16"), (6, 2, 64, 32, "e4m3"), (16, 2, 128, 8, "e4m3"),
                                               (3, 3, 64, 64, "bf16")])
@pytest.mark.parametrize("new,ctx,groups", PREFIX)
def test_attention_prefix(bd, new, ctx, groups, H, Hk, D, page, cache):
    Case(new, ctx, H, Hk, D, page, cache, groups=groups, pad=1, seed=len(new)).check(bd)


@pytest.mark.parametrize("max_new", [0, 1, 5, 1000])
def test_attention_hint_does_not_matter(bd, max_new):
    """A wrong or missing max_new gives the same answers (within the bounds)."""
    Case([1, 37, 2], [40, 3, 100], 8, 2, 128, 16, seed=2, max_new=max_new).check(bd)


def test_attention_rows_without_keys(bd):
    """Sequences shorter than their new tokens, empty tables of pages, no sequence at all."""
    for new in ([4, 1, 2], [40, 1, 2]):
        c = Case(new, [0, 0, 5], 8, 2, 128, 16, seed=1)
        c.host.kv_len = np.array([2, 0, 7])            # the first tokens of sequence 0 and all of 1 see nothing
        c.host.table[2, 0] = -1                        # and 2 has lost its page
        out = c.check(bd)
        assert not out[:new[0] - 2].any() and not out[new[0]].any() and not out[new[0] + 1:].any()
    c = Case([], [], 8, 2, 64, 16, pad=3, fill=False, max_new=0)
    b = bd.PagedBatch(i32([0]), i32(np.zeros(0)), i32(np.zeros((0, 1))))
    assert not bd.attention(c.q, c.kv(bd), b).any()
    assert bd.attention(c.q[:0], c.kv(bd), b).shape == (0, 8, 64)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[1, 2, 1], [50, 2, 33], [150, 20, 70]])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attention_bad_pages_lengths_and_starts(bd, new, cache, D):
    """Page numbers out of range hold no key, lengths end with the table, starts with the tokens."""
    c = Case(new, [100, 40, 77], 8, 2, D, 16, cache, groups=[(0, 3, 90)], seed=4)
    c.host.table[0, 2], c.host.table[1, 0], c.host.table[2, 1] = -1, c.n_pages, 2 ** 31 - 1
    c.host.ptable[0, [0, 3]] = -2 ** 31, c.n_pages + 5
    c.check(bd)
    b = c.batch(bd)
    want = bd.attention(c.q, c.kv(bd), b)
    wide = i32(np.concatenate([c.host.q_start[:-1], [10 ** 9]]))
    longer = bd.PagedBatch(wide, b.kv_len, b.page_table, group_start=i32([-5, 10 ** 6]), prefix_len=b.prefix_len,
                           prefix_table=b.prefix_table, max_new=c.max_new)
    assert torch.equal(bd.attention(c.q, c.kv(bd), longer), want)
    full = c.host.kv_len.copy()
    full[2] = c.host.table.shape[1] * 16
    c2 = bd.PagedBatch(b.q_start, i32(full), b.page_table, max_new=c.max_new)
    full[2] = 2 ** 31 - 1
    c3 = bd.PagedBatch(b.q_start, i32(full), b.page_table, max_new=c.max_new)
    c.k.view(torch.uint8).zero_()
    c.v.view(torch.uint8).zero_()
    assert torch.equal(bd.attention(c.q, c.kv(bd), c2), bd.attention(c.q, c.kv(bd), c3))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,ctx", [([2, 3], [20, 40]), ([70, 3], [9, 40]), ([200, 3], [190, 40])])
def test_attention_later_keys_do_not_reach_earlier_rows(bd, new, ctx, D):
    """NaN and infinities in a key or value show in the tokens that see it and in no other."""
    for which, bad in (("k", NAN), ("v", NAN), ("v", float("inf")), ("v", -float("inf")), ("k", float("inf"))):
        c = Case(new, ctx, 8, 2, D, 16, seed=6)
        want = bd.attention(c.q, c.kv(bd), c.batch(bd)).clone()
        at = ctx[0] + new[0] - 1                        # the last token's own cell
        pg = int(c.host.table[0, at // 16])
        getattr(c, which)[pg, 0, at % 16, 5] = bad
        got = bd.attention(c.q, c.kv(bd), c.batch(bd))
        keep = torch.ones(c.T, dtype=torch.bool)
        keep[new[0] - 1] = False
        assert torch.equal(got[keep], want[keep]), (which, bad)
        assert torch.equal(got[new[0] - 1, 4:], want[new[0] - 1, 4:])
        if which == "v":
            assert not got[new[0] - 1, :4, 5].isfinite().any()
            rest = [i for i in range(D) if i != 5]
            assert torch.equal(got[new[0] - 1, :4, rest], want[new[0] - 1, :4, rest])


def test_attention_large_scores(bd):
    """Scores of several thousand: the running maximum keeps every exponent in range."""
    c = Case([1, 40], [700, 100], 8, 2, 128, 16, seed=8)
    c.check(bd, scale=40.0)
    c.check(bd, scale=1e-6)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attention_long_prompt_and_context(bd, cache):
    """Many plain steps, splits of one sequence's keys, and a bad page in the middle of them."""
    c = Case([3, 140], [700, 1900], 4, 1, 128, 32, cache, seed=31)
    c.host.table[1, 20] = -1
    c.check(bd)
    c = Case([260], [1500], 3, 1, 64, 64, cache, groups=[(0, 1, 500)], seed=32)
    c.check(bd)


def test_attention_strided_q_and_out(bd):
    c = Case([1, 1, 30], [50, 3, 90], 8, 2, 128, 16, seed=12)
    wide = torch.zeros(c.T, 8 * 128 + 40, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 8:8 + 1024].unflatten(1, (8, 128))
    q.copy_(c.q)
    want = c.check(bd)
    out = torch.full_like(want, NAN)
    assert bd.attention(q, c.kv(bd), c.batch(bd), out=out) is out
    assert torch.equal(out, want)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_cache_beyond_32_bit_offsets(bd, cache):
    """A cache of more than 4 GiB a side: the last pages are its own, not a wrapped offset's."""
    dt, page, Hk, D = (torch.bfloat16, 64, 8, 128) if cache == "bf16" else (torch.float8_e4m3fn, 128, 8, 128)
    n_pages = (9 << 30) // 2 // (page * Hk * D * (2 if cache == "bf16" else 1))
    kv = bd.PagedKV.empty(n_pages, Hk, page, D, dt)
    pages = [n_pages - 1, 0, n_pages - 2, n_pages // 2]
    c = Case([2, 70], [100, 30], 16, Hk, D, page, cache, seed=3, fill=False)
    small = np.unique(c.host.table[c.host.table < c.n_pages])
    assert len(small) <= len(pages)
    table = c.host.table.copy()
    for a, b in zip(small, pages):
        kv.k[b].copy_(c.k[a])
        kv.v[b].copy_(c.v[a])
        table[c.host.table == a] = b
    b = c.batch(bd)
    want = bd.attention(c.q, bd.PagedKV(c.k, c.v), b)
    got = bd.attention(c.q, kv, bd.PagedBatch(b.q_start, b.kv_len, i32(table), max_new=70))
    assert torch.equal(got, want)
    # and the append reaches them
    g = gen(4)
    k, v = randn(g, 72, Hk, D).to(DEV), randn(g, 72, Hk, D).to(DEV)
    bd.kv_append(None, k, v, None, kv, bd.PagedBatch(b.q_start, b.kv_len, i32(table)))
    ck = bd.PagedKV(c.k, c.v)
    bd.kv_append(None, k, v, None, ck, b)
    for a, p in zip(small, pages):
        assert torch.equal(kv.k[p].view(torch.uint8), c.k[a].view(torch.uint8))
        assert torch.equal(kv.v[p].view(torch.uint8), c.v[a].view(torch.uint8))


# ------------------------------------------------------------------- append

APPENDS = [  # new, ctx, H, Hk, D, page, rotary, groups
    ([1], [0], 1, 1, 64, 1, 64, []), ([1, 1, 1], [0, 15, 16], 8, 2, 128, 16, 128, []),
    ([5, 0, 33], [7, 3, 0], 6, 3, 64, 8, 32, [(0, 3, 1000003)]), ([2, 1, 70], [60, 5, 0], 16, 2, 128, 64, 16, [(0, 1, 9), (1, 3, 70)]),
    ([600, 7], [0, 1], 2, 1, 128, 32, 64, []), ([3], [2], 4, 4, 128, 2, 0, []),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,ctx,H,Hk,D,page,rotary,groups", APPENDS)
def test_kv_append(bd, new, ctx, H, Hk, D, page, rotary, groups, interleaved, cache):
    far = [(a, b, min(p, 100)) for a, b, p in groups]
    c = Case(new, ctx, H, Hk, D, page, cache, groups=far, pad=2, seed=H + D, fill=False)
    if groups:                                         # the append reads no prefix page, only its length
        c.host.prefix_len = [p for _, _, p in groups]
        c.host.ptable = np.zeros((len(groups), max(p for _, _, p in groups) // page + 1), np.int32)
    g = gen(7)
    fused = randn(g, c.T, (H + 2 * Hk) * D).to(DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in fused.split([H * D, Hk * D, Hk * D], 1))
    inv = torch.tensor(10000.0, dtype=torch.float64) ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1))
    before = [t.view(torch.uint8).clone() for t in (c.k, c.v)]
    b = c.batch(bd)
    got = bd.kv_append(q, k, v, inv.to(DEV) if rotary else None, c.kv(bd), b, interleaved=interleaved)
    wq, tq = np.zeros((c.T, H, D)), np.zeros((c.T, H, D))
    wk, wv = c.values() if cache == "bf16" else (f64(c.k), f64(c.v))
    wk, wv, tk, tv = wk.copy(), wv.copy(), np.zeros_like(wk), np.zeros_like(wv)
    touched = np.zeros((c.n_pages, page), bool)
    half = ref.BF if cache == "bf16" else ref.E4
    sub = 0.0 if cache == "bf16" else 2.0 ** -10
    for t in range(c.T):
        pl = c.host.place(t)
        if pl is None:
            continue
        s, at, gi, p = pl
        y, mag = ref.rotate(f64(q[t]), at + p, inv.numpy(), interleaved)
        wq[t], tq[t] = y, ref.BF * (np.abs(y) + 2.0 ** -20 * mag) + 2.0 ** -20 * mag
        pg, sl = c.host.cell(c.host.table[s], at)
        touched[pg, sl] = True
        y, mag = ref.rotate(f64(k[t]), at + p, inv.numpy(), interleaved)
        z = f64(v[t])
        ks = vs = np.ones((Hk, 1))
        if cache == "e4m3":
            ks, vs = f64(c.k_scale)[:, None], f64(c.v_scale)[:, None]
        for w, tol, val, m, sc in ((wk, tk, y, mag, ks), (wv, tv, z, np.abs(z), vs)):
            e = 2.0 ** -20 * m / sc
            lim = np.inf if cache == "bf16" else 448.0
            w[pg, :, sl] = np.clip(val / sc, -lim, lim)
            tol[pg, :, sl] = half * (np.abs(w[pg, :, sl]) + e) + e + sub
    close(got, wq, tq, "q")
    close(c.k, wk, tk, "k")
    close(c.v, wv, tv, "v")
    un = torch.from_numpy(~touched).to(DEV)[:, None, :, None].expand(c.k.shape)
    for t, old in zip((c.k, c.v), before):
        new_b = t.view(torch.uint8).view(*c.k.shape[:3], -1)
        m = un[..., :1].expand(new_b.shape)
        assert torch.equal(new_b[m], old.view(new_b.shape)[m])


def test_kv_append_in_place_values_and_bad_pages(bd):
    """q in place, saturation and NaN in 8 bits, tokens whose page is gone, far positions without a float's angle."""
    c = Case([1, 1, 2], [3, 20, 40], 4, 2, 64, 16, "e4m3", seed=1, fill=False)
    g = gen(2)
    q, k, v = randn(g, 4, 4, 64).to(DEV), randn(g, 4, 2, 64).to(DEV), randn(g, 4, 2, 64).to(DEV)
    v[0, 0, 0], v[0, 0, 1], v[0, 0, 2], v[0, 0, 3] = 1e4, -1e4, NAN, float("inf")
    c.host.table[1, 1] = -3
    inv = torch.full((32,), 1.0, dtype=torch.float64, device=DEV)
    kv, b = c.kv(bd), c.batch(bd)
    old = c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()
    want = bd.kv_append(q, k, v, inv, kv, b)
    assert bd.kv_append(q, k, v, inv, kv, b, q_out=q) is q
    assert torch.equal(q, want)
    cell = f64(c.v[int(c.host.table[0, 0]), 0, 3, :4])
    assert cell[0] == 448 and cell[1] == -448 and np.isnan(cell[2]) and cell[3] == 448
    lost = [p for p in range(c.n_pages) if p not in c.host.table]
    for t, o in zip((c.k, c.v), old):
        assert torch.equal(t.view(torch.uint8)[lost], o.view(t.shape)[lost])
        assert torch.equal(t.view(torch.uint8)[int(c.host.table[1, 0])], o.view(t.shape)[int(c.host.table[1, 0])])
    c.host.kv_len[0] = 0                              # a token at a place below 0: no cell, a zero query
    out = bd.kv_append(q, k, v, inv, kv, c.batch(bd))
    assert not out[0].any() and out[1].any()


# ----------------------------------------------------------- together, streams


def test_another_stream_and_graph_replays(bd):
    """Append then attention captured once and replayed while the lengths, tables and inputs change in place."""
    c = Case([1, 1, 1, 1], [40, 3, 100, 64], 16, 2, 128, 16, groups=[(0, 2, 50)], seed=11)
    g = gen(5)
    kv, b = c.kv(bd), c.batch(bd)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).to(DEV)
    q, k, v = randn(g, 4, 16, 128).to(DEV), randn(g, 4, 2, 128).to(DEV), randn(g, 4, 2, 128).to(DEV)
    res, w = randn(g, 4, 2048).to(DEV), randn(g, 3, 2048).to(DEV)
    ids = torch.tensor([0, 2, 1, 0], dtype=torch.int32, device=DEV)

    def step():
        rq = bd.kv_append(q, k, v, inv, kv, b)
        o = bd.attention(rq, kv, b)
        return (rq, o) + bd.block_norm(res, o.view(4, 2048), post_weight=w, pre_weight=w, variant_ids=ids)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        for t in (q, k, v):
            t.copy_(randn(g, *t.shape).to(DEV))
        b.kv_len.copy_(i32([41 - 9 * i, 4, 101 - i, 65 - 20 * i]))
        graph.replay()
        torch.cuda.synchronize()
        for a, w_ in zip(got, step()):
            assert torch.equal(a, w_), i
        torch.cuda.synchronize()


def test_same_bits_every_time(bd):
    """No atomics: two runs give the same bits."""
    c = Case([1] * 7 + [90], [700, 3, 64, 900, 0, 31, 2000, 100], 16, 2, 128, 16, groups=[(0, 5, 300)], seed=21, fill=False)
    a = bd.attention(c.q, c.kv(bd), c.batch(bd))
    for _ in range(3):
        assert torch.equal(bd.attention(c.q, c.kv(bd), c.batch(bd)), a)
