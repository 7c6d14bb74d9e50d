"""GPU tier: the operators between a hidden state and the next token together: the
attention half of a layer over an 8-bit base, the head and the draw, against the
same in 64 bits; a loop of decoding steps, each token the next step's input, run
eagerly and replayed from a captured graph; streams other than the default one."""
import numpy as np
import pytest
import torch

from tests import decoder_ref as ref
from tests import int8_ref, sample_ref

pytestmark = pytest.mark.gpu

V, D, H, HK, DM, PAGE, VOCAB = 3, 64, 4, 2, 256, 16, 5003


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def layer(bd, rows, cols, seed):
    """A projection over an 8-bit base, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    w, c = bd.quantize_int8(torch.randn(rows, cols, generator=g).mul_(cols ** -0.5).cuda())
    signs = torch.randint(0, 256, (V, rows, cols // 8), generator=g, dtype=torch.uint8).cuda()
    alpha = (torch.rand(V, rows, generator=g) * 0.2 * cols ** -0.5).cuda()
    return w, c, signs, alpha


class Model:
    """One attention half and the head, the parts that a decoding step goes through."""

    def __init__(self, bd, seed=1):
        from tenant_fine_tune_amd.block import AttentionBlock, OutputBlock

        g = torch.Generator().manual_seed(seed)
        self.bd = bd
        self.qkv, self.out = layer(bd, (H + 2 * HK) * D, DM, seed), layer(bd, DM, H * D, seed + 1)
        self.post, self.nxt = ((1 + torch.randn(V, DM, generator=g) * 0.2).to(torch.bfloat16).cuda() for _ in range(2))
        self.inv = torch.tensor(10000.0, dtype=torch.float64) ** (-torch.arange(32, dtype=torch.float64) / 32)
        self.kv = bd.PagedKV.empty(24, HK, PAGE, D)
        self.kv.k.zero_()
        self.kv.v.zero_()
        self.attention = AttentionBlock(self.qkv, self.out, H, self.kv, self.inv.cuda(), post_weight=self.post,
                                        next_weight=self.nxt, scale=0.5)
        self.embed = torch.randn(VOCAB, DM, generator=g).to(torch.bfloat16).cuda()
        self.head = bd.quantize_int8(self.embed)
        self.output = OutputBlock(self.head)

    def step(self, tokens, ids, batch, u, rows=None, **settings):
        x = self.embed.index_select(0, tokens)
        _, normed = self.bd.block_norm(x, pre_weight=self.nxt, variant_ids=ids)
        x, _ = self.attention.forward(normed, x.float(), ids, batch)
        return x, *self.output.forward(x, u, rows, **settings)


def bf(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double()


def linear64(x, ids, l):
    """x bf16 values in 64 bits; (the product from the rows in 8 bits, a row's step relative to its rms)."""
    q, s = int8_ref.quantized(x.to(torch.bfloat16))
    y, _ = int8_ref.linear(q, s, *(t.cpu() for t in l), ids)
    return bf(y), (s.double() / x.pow(2).mean(-1).sqrt()).max().item()


def test_prompts_to_tokens_against_64_bits(bd):
    m = Model(bd)
    g = torch.Generator().manual_seed(5)
    lens, owner = [21, 1, 9], [2, 0, 1]
    T = sum(lens)
    tokens = torch.randint(0, VOCAB, (T,), generator=g)
    ids = torch.repeat_interleave(torch.tensor(owner), torch.tensor(lens)).int()
    starts = np.concatenate([[0], np.cumsum(lens)])
    rows = torch.tensor(starts[1:] - 1)
    u = torch.rand(3, generator=g)
    temperature, top_k, top_p, min_p = torch.tensor([0.7, 1.0, 2.0]), torch.tensor([0, 40, 0]).int(), \
        torch.tensor([0.9, 1.0, 1.0]), torch.tensor([0.0, 0.0, 0.01])
    batch = bd.PagedBatch(i32(starts.tolist()), i32(lens), i32([[5, 9], [8, 0], [1, 2]]))
    x, got, logprobs = m.step(tokens.cuda(), ids.cuda(), batch, u.cuda(), rows.cuda(), temperature=temperature.cuda(),
                              top_k=top_k.cuda(), top_p=top_p.cuda(), min_p=min_p.cuda())

    e = m.embed.double().cpu()[tokens]
    _, normed, _, _ = ref.block_norm(e.numpy(), None, None, None, "none", 1.0, m.nxt.double().cpu().numpy(), ids.numpy(), 1e-6)
    fused, _ = linear64(bf(normed), ids, m.qkv)
    fused = fused.numpy()
    q, k, v = (t.reshape(T, -1, D) for t in np.split(fused, [H * D, (H + HK) * D], 1))
    o = np.zeros((T, H, D))
    for s in range(3):
        at = range(starts[s], starts[s + 1])
        kk = np.stack([bf(ref.rotate(k[t], t - starts[s], m.inv.numpy(), False)[0]).numpy() for t in at])
        for t in at:
            qt = bf(ref.rotate(q[t], t - starts[s], m.inv.numpy(), False)[0]).numpy()
            n = t - starts[s] + 1
            for h in range(H):
                z = kk[:n, h // 2] @ qt[h] / np.sqrt(D)
                w = np.exp(z - z.max())
                o[t, h] = w @ v[starts[s]:starts[s] + n, h // 2] / w.sum()
    y, step = linear64(bf(o.reshape(T, -1)), ids, m.out)
    want, xn, _, _ = ref.block_norm(e.numpy(), y.numpy(), m.post.double().cpu().numpy(), None, "none", 0.5,
                                    m.nxt.double().cpu().numpy(), ids.numpy(), 1e-6)
    err = x.double().cpu().numpy() - xn
    # the first norm, q/k/v, rotation, attention and the block's output are rounded to bf16
    # (2^-8 at most each); where these move a number over a border in front of a projection it
    # moves by one step of the row there (two projections, `step` of the row's rms at most)
    bound = (6 * 2.0 ** -16 + 2 * step ** 2) ** 0.5
    assert np.sqrt((err ** 2).mean()) <= bound * np.sqrt((xn ** 2).mean())

    # from the block's own output on: the logits' sums are exact, each token is one that 64 bits allow
    q, s = int8_ref.quantized(x[rows.cuda()].cpu())
    logits, size = int8_ref.linear(q, s, *(t.cpu() for t in m.head))
    mine = m.output.logits(x, rows.cuda())
    int8_ref.check(mine, logits, size)
    sample_ref.check(got, logprobs, mine, u, temperature, top_k, top_p, min_p)


SETTINGS = dict(temperature=0.8, top_k=50, top_p=0.95)


def decode(m, state, out):
    """One step of three sequences in place: the tokens drawn are the next ones."""
    batch = m.bd.PagedBatch(state["start"], state["lens"], state["pages"], max_new=1)
    u = state["u"].index_select(0, state["at"])[0]
    _, tokens, logprobs = m.step(state["tokens"], state["ids"], batch, u, **SETTINGS)
    out[0].copy_(tokens)
    out[1].copy_(logprobs)
    state["tokens"].copy_(tokens)
    state["lens"].add_(1)
    state["at"].add_(1)


def begin(steps, seed=9):
    g = torch.Generator().manual_seed(seed)
    return dict(start=i32([0, 1, 2, 3]), lens=i32([1, 1, 1]), pages=i32([[5, 9], [8, 0], [1, 2]]), ids=i32([1, 0, 2]),
                tokens=torch.randint(0, VOCAB, (3,), generator=g).cuda(), at=torch.zeros(1, dtype=torch.int64, device="cuda"),
                u=torch.rand(steps, 3, generator=g).cuda())


def test_decoding_loop_eager_and_replayed(bd):
    steps = 20
    m = Model(bd)
    out = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, device="cuda")
    state, eager = begin(steps), []
    for _ in range(steps):
        decode(m, state, out)
        eager.append((out[0].cpu(), out[1].cpu()))
    assert all(((t >= 0) & (t < VOCAB)).all() and torch.isfinite(p).all() for t, p in eager)

    state = begin(steps)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(m, {k: v.clone() for k, v in state.items()}, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode(m, state, out)
    again = begin(steps)
    for k in state:
        state[k].copy_(again[k])
    other = torch.randn(70, 256, device="cuda")
    for tokens, logprobs in eager:
        graph.replay()
        assert torch.equal(out[0].cpu(), tokens) and torch.equal(out[1].cpu(), logprobs)
        m.output.forward(other.bfloat16(), torch.rand(70, device="cuda"))     # eager work between the replays
        torch.cuda.synchronize()


def calls(bd, seed, m):
    """The three operators with workspaces, over the kernels that m picks; inputs of a seed."""
    c = [t.cuda() if t is not None else None for t in int8_ref.random_case(m, 600, 4096, 3, seed)]
    x = torch.randn(m, 4096, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    u = torch.rand(m, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + 1))

    def run():
        q, s = bd.quantize_int8(x)
        y = bd.linear_int8(q, s, *c[2:6], variant_ids=c[6], out_dtype=torch.float32)
        return q, s, y, *bd.sample(y, u, top_p=0.9, temperature=0.5)

    return run


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("m", [3, 40, 300])
def test_two_streams_at_once(bd, m):
    runs = [calls(bd, seed, m) for seed in (1, 2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for _ in range(10):
        for i, (r, s) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(s):
                got[i].append(r())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(g, want[i]) for g in got[i])


@pytest.mark.parametrize("m", [3, 40, 300])
def test_two_graphs_in_turn(bd, m):
    runs = [calls(bd, seed, m) for seed in (3, 4)]
    want = [r() for r in runs]
    pool = torch.cuda.graph_pool_handle()
    graphs, got = [], []
    for r in runs:      # of one pool: the second's workspaces may lie where the first's did
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            got.append(r())
        graphs.append(graph)
    for _ in range(4):
        for i in (0, 1):
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(got[i], want[i])
            runs[1 - i]()


@pytest.mark.parametrize("m", [17, 100, 300])
def test_one_workspace_for_many_calls(bd, m):
    """A caller's own scratch, dirty from the call before and longer than asked for, through the C entries."""
    q, s, w, c, signs, alpha, ids = (t.cuda() for t in int8_ref.random_case(m, 600, 4096, 3, 7))
    need = max(bd.lib.bitdelta_linear_int8_workspace(m, 3, 600, 4096), bd.lib.bitdelta_sample_workspace(m, 600))
    work = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    want = bd.linear_int8(q, s, w, c, signs, alpha, variant_ids=ids, out_dtype=torch.float32)
    u = torch.rand(m, device="cuda")
    drawn = bd.sample(want, u)
    for _ in range(3):
        y, t, p = torch.empty_like(want), torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty(m, device="cuda")
        assert bd.lib.bitdelta_linear_int8(q.data_ptr(), s.data_ptr(), m, w.data_ptr(), c.data_ptr(), signs.data_ptr(),
                                           alpha.data_ptr(), bd.BD_ALPHA_ROW, ids.data_ptr(), 3, 600, 4096, y.data_ptr(),
                                           bd.BD_F32, work.data_ptr(), need, stream) == bd.BD_OK
        assert bd.lib.bitdelta_sample(y.data_ptr(), 600, bd.BD_F32, m, 600, u.data_ptr(), 0, 1.0, 0, 0, 0, 1.0, 0, 0.0,
                                      t.data_ptr(), p.data_ptr(), work.data_ptr(), need, stream) == bd.BD_OK
        assert torch.equal(y, want) and torch.equal(t, drawn[0]) and torch.equal(p, drawn[1])
    assert (work[need:] == 0xAB).all()
