"""GPU tier: rows in 8 bits and products over an 8-bit base against their
definitions in 64 bits (tolerances: tests/int8_ref.py)."""
import pytest
import torch

from tests import int8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bd():
    import tenant_fine_tune_amd as bd

    return bd


def quantize_matches(bd, x, **kw):
    q, s = bd.quantize_int8(x, **kw)
    rq, rs = ref.quantized(x)
    assert q.dtype == torch.int8 and s.dtype == torch.float32 and q.shape == x.shape and s.shape == x.shape[:-1]
    assert torch.equal(s.cpu().nan_to_num(-1.0), rs.nan_to_num(-1.0))
    assert torch.equal(q.cpu(), rq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,d", [(1, 1), (3, 7), (5, 8), (70, 63), (2, 513), (9, 2048), (4, 2049), (33, 8192), (2, 16391),
                                 (3, 28672), (2, 32768), (2, 32769), (1, 65537), (1, 131064)])
def test_quantize(bd, m, d, dtype):
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(m, d, generator=g) * torch.exp(torch.randn(m, 1, generator=g))).to(dtype)
    quantize_matches(bd, x.to(DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_ties_and_borders(bd, dtype):
    # rows whose scale is a power of two times odd numbers: every half is met, from both sides
    rows = []
    for odd in (1, 3, 5, 7, 11):
        half = (torch.arange(254, dtype=torch.float64) - 127 + 0.5) * odd
        rows.append(torch.cat([half, torch.tensor([127.0 * odd, -127.0 * odd])]))
    x = torch.stack(rows).float()
    up, down = torch.nextafter(x, torch.tensor(1e9)), torch.nextafter(x, torch.tensor(-1e9))
    x = torch.cat([x, up, down]).clamp(-127 * 11, 127 * 11).to(dtype).to(DEV)
    for scale in (1.0, 2.0 ** -90, 2.0 ** 60):
        quantize_matches(bd, x * scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [2.0 ** -149, 2.0 ** -144, 2.0 ** -142, 2.0 ** -130, 2.0 ** -120, 2.0 ** -101, 3e38])
def test_quantize_tiny_and_huge(bd, size, dtype):
    g = torch.Generator().manual_seed(3)
    x = (torch.rand(4, 300, generator=g, dtype=torch.float64) * 2 - 1) * size
    quantize_matches(bd, x.to(dtype).to(DEV))


def test_quantize_rows_that_are_not_numbers(bd):
    x = torch.randn(6, 70)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 69] = float("inf")
    x[3, 0] = float("-inf")
    x[4, 5:7] = torch.tensor([float("inf"), float("nan")])
    for dtype in (torch.bfloat16, torch.float32):
        quantize_matches(bd, x.to(dtype).to(DEV))


def test_quantize_strides_shapes_and_outputs(bd):
    x = torch.randn(12, 50, device=DEV)
    quantize_matches(bd, x[:, :33])
    quantize_matches(bd, x[::3, 1:42])
    quantize_matches(bd, x.bfloat16()[1:2, 5:])
    quantize_matches(bd, x.view(3, 4, 50))
    quantize_matches(bd, x[0])
    q, s = torch.full((14, 50), 99, dtype=torch.int8, device=DEV), torch.full((14,), 9.0, device=DEV)
    quantize_matches(bd, x, out=q[1:13], scale_out=s[1:13])
    assert (q[[0, 13]] == 99).all() and (s[[0, 13]] == 9).all()
    q, s = bd.quantize_int8(x[:0])
    assert q.shape == (0, 50) and s.shape == (0,)


def run(bd, c, **kw):
    q, s, w, ws, signs, alpha, ids = (t.to(DEV) if t is not None else None for t in c)
    return bd.linear_int8(q, s, w, ws, signs, alpha, variant_ids=ids, **kw)


def linear_matches(bd, c, **kw):
    y = run(bd, c, **kw)
    r, size = ref.linear(*c)
    assert y.shape == r.shape
    ref.check(y, r, size)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 129, 300])
@pytest.mark.parametrize("variants", [0, 1, 5])
def test_linear_tokens(bd, m, variants):
    linear_matches(bd, ref.random_case(m, 96, 640, variants, m), out_dtype=torch.float32)


@pytest.mark.parametrize("k", [8, 16, 24, 32, 40, 64, 72, 96, 128, 136, 192, 248, 256, 448, 512, 520, 576, 1024, 1032,
                               4096, 4104, 4160, 8192])
@pytest.mark.parametrize("m", [3, 70])
def test_linear_widths(bd, k, m):
    for variants in (0, 1, 3):
        linear_matches(bd, ref.random_case(m, 33, k, variants, k), out_dtype=torch.float32)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 64, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("m", [1, 20, 70, 260])
def test_linear_channels(bd, n, m):
    linear_matches(bd, ref.random_case(m, n, 256, 3, n), out_dtype=torch.float32)
    linear_matches(bd, ref.random_case(m, n, 320, 1, n), out_dtype=torch.bfloat16)


@pytest.mark.parametrize("variants", [2, 14, 64, 300])
@pytest.mark.parametrize("m", [1, 16, 40, 64, 130, 700])
@pytest.mark.parametrize("per_matrix", [False, True])
def test_linear_variants(bd, variants, m, per_matrix):
    c = ref.random_case(m, 48, 512, variants, m + variants, per_matrix)
    linear_matches(bd, c, per_matrix=per_matrix)


@pytest.mark.parametrize("m", [4, 30, 64, 150])
def test_linear_ids_outside(bd, m):
    c = ref.random_case(m, 40, 256, 3, 5)
    c[6][::3] = torch.tensor([-1, 3, 2 ** 31 - 1, -2 ** 31])[torch.arange(len(c[6][::3])) % 4].int()
    linear_matches(bd, c)
    c[6][:] = 7
    assert (run(bd, c) == 0).all()


@pytest.mark.parametrize("m", [2, 40, 90])
def test_linear_extreme_numbers(bd, m):
    # the largest sums: every product 2^14, over the widest rows
    n, k = 18, 131064
    q, w = torch.full((m, k), -128, dtype=torch.int8), torch.full((n, k), -128, dtype=torch.int8)
    w[1::2] = 127
    signs = torch.full((n, k // 8), 255, dtype=torch.uint8)
    signs[::3] = 0
    c = (q, torch.ones(m), w, torch.ones(n), signs, torch.full((n,), 0.5), None)
    linear_matches(bd, c, out_dtype=torch.float32)
    linear_matches(bd, ref.random_case(m, n, 4096, 2, 1, extremes=True), out_dtype=torch.float32)


@pytest.mark.parametrize("m", [5, 80])
@pytest.mark.parametrize("slip", [1, 2, 3, 4])
def test_linear_signs_of_any_alignment(bd, m, slip):
    for k in (256, 72):
        for variants in (1, 3):
            q, s, w, ws, signs, alpha, ids = ref.random_case(m, 21, k, variants, slip)
            room = torch.zeros(signs.numel() + 8, dtype=torch.uint8, device=DEV)
            at = room[slip:slip + signs.numel()].view(signs.shape)
            at.copy_(signs)
            y = bd.linear_int8(q.to(DEV), s.to(DEV), w.to(DEV), ws.to(DEV), at, alpha.to(DEV),
                               variant_ids=None if ids is None else ids.to(DEV), out_dtype=torch.float32)
            ref.check(y, *ref.linear(q, s, w, ws, signs, alpha, ids))


def test_linear_scales(bd):
    q, s, w, ws, signs, alpha, _ = ref.random_case(6, 24, 128, 1, 1)
    s[0], s[1], s[2] = 0.0, -1.0, 1e-30
    ws[3], ws[4], alpha[5], alpha[6] = 0.0, -2.0, 0.0, -1.0
    linear_matches(bd, (q, s, w, ws, signs, alpha, None), out_dtype=torch.float32)
    s[3] = float("nan")
    y = run(bd, (q, s, w, ws, signs, alpha, None))
    assert y[3].isnan().all() and not y[[0, 1, 2, 4, 5]].isnan().any()


def test_linear_cancelling_sums(bd):
    # base and delta cancel all but a small rest, which stays exact
    q, s, w, ws, signs, alpha, _ = ref.random_case(9, 16, 8192, 1, 4)
    w[:] = 1 - 2 * (1 - ((signs[..., None] >> torch.arange(8, dtype=torch.uint8)) & 1).flatten(-2).to(torch.int8))
    ws[:], alpha[:] = 1.0, -1.0 - 2.0 ** -23
    linear_matches(bd, (q, s, w, ws, signs, alpha, None), out_dtype=torch.float32)


def test_linear_shapes_and_outputs(bd):
    c = ref.random_case(12, 40, 64, 1, 2)
    q, s, w, ws, signs, alpha, _ = (t.to(DEV) if t is not None else None for t in c)
    y = bd.linear_int8(q.view(3, 4, 64), s.view(3, 4), w, ws, signs, alpha)
    assert y.shape == (3, 4, 40) and torch.equal(y.view(12, 40), bd.linear_int8(q, s, w, ws, signs, alpha))
    out = torch.full((14, 40), 7.0, device=DEV)
    assert bd.linear_int8(q, s, w, ws, signs, alpha, out=out[1:13]).data_ptr() == out[1:13].data_ptr()
    assert (out[[0, 13]] == 7).all()
    ref.check(out[1:13], *ref.linear(*c))
    assert bd.linear_int8(q[:0], s[:0], w, ws).shape == (0, 40)
    assert bd.linear_int8(q[0], s[0], w, ws).shape == (40,)


@pytest.mark.parametrize("m", [1, 16, 50, 64, 200])
def test_linear_tokens_do_not_depend_on_each_other(bd, m):
    c = ref.random_case(300, 64, 1536, 6, 11)
    whole = run(bd, c, out_dtype=torch.float32)
    part = run(bd, (c[0][100:100 + m], c[1][100:100 + m], *c[2:6], c[6][100:100 + m]), out_dtype=torch.float32)
    assert torch.equal(part, whole[100:100 + m])


def test_linear_of_quantized_rows_is_near_the_product(bd):
    """The use: |y - x W^T| is within the two roundings, half a step of each row's scale."""
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(20, 512, generator=g).bfloat16(), (torch.randn(70, 512, generator=g) * 0.02).bfloat16()
    q, s = bd.quantize_int8(x.to(DEV))
    c, cs = bd.quantize_int8(w.to(DEV))
    y = bd.linear_int8(q, s, c, cs, out_dtype=torch.float32).cpu().double()
    x, w = x.double(), w.double()
    dx, dw = s.cpu().double()[:, None] / 2, cs.cpu().double()[:, None] / 2
    bound = dx * w.abs().sum(1) + x.abs().sum(1)[:, None] * dw.T + 512 * dx * dw.T
    assert ((y - x @ w.T).abs() <= bound * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("variants", [0, 3])
def test_linear_more_tokens_than_a_launch_takes(bd, variants):
    # rows that end inside 32 columns and too many to copy: slices, the last of them short
    for m in ((1 << 23) + 5, (1 << 23) + (1 << 20) + 40):
        linear_matches(bd, ref.random_case(m, 2, 8, variants, 3), out_dtype=torch.float32)


@pytest.mark.parametrize("m", [65, 100, 128, 129, 192, 300])
@pytest.mark.parametrize("variants", [13, 40, 200])
def test_linear_many_variants_in_lots(bd, m, variants):
    linear_matches(bd, ref.random_case(m, 130, 1056, variants, m), out_dtype=torch.float32)


@pytest.mark.parametrize("m,n,k", [(70, 130, 40), (333, 1000, 4104), (130, 257, 1032), (65, 1, 8), (90, 64, 8200)])
@pytest.mark.parametrize("variants", [0, 1, 3, 16])
def test_linear_rows_that_end_inside_32_columns(bd, m, n, k, variants):
    linear_matches(bd, ref.random_case(m, n, k, variants, k), out_dtype=torch.float32)
    linear_matches(bd, ref.random_case(m, n, k, variants, k + 1, extremes=True))


@pytest.mark.parametrize("m,n,k", [(80, 2048, 8192), (512, 512, 16384), (1000, 300, 8192), (200, 4096, 2048)])
@pytest.mark.parametrize("variants", [0, 1, 3])
def test_linear_split_columns(bd, m, n, k, variants):
    linear_matches(bd, ref.random_case(m, n, k, variants, m), out_dtype=torch.float32)
