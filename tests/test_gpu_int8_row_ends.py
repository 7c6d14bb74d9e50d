"""GPU tier: products over an 8-bit base whose rows end anywhere inside 32 columns, from one
step of columns to split ones, with the base in the middle of other numbers."""
import pytest
import torch

from tests import int8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("m", [66, 200])
@pytest.mark.parametrize("k", [8, 16, 24, 40, 48, 56, 120, 128, 136, 144, 152, 264, 1000, 1032, 1048, 4120, 8200, 8216])
def test_rows_that_end_anywhere(k, m):
    import tenant_fine_tune_amd as bd

    n = 131
    for variants in (0, 1, 3):
        for per_matrix in (False, True) if variants else (False,):
            c = ref.random_case(m, n, k, variants, k + m, per_matrix, extremes=True)
            q, s, w, ws, signs, alpha, ids = (None if t is None else t.to(DEV) for t in c)
            room = torch.full((n + 3, k), -128, dtype=torch.int8, device=DEV)
            at = room[2:n + 2]
            at.copy_(w)
            y = bd.linear_int8(q, s, at, ws, signs, alpha, variant_ids=ids, per_matrix=per_matrix if variants else None,
                               out_dtype=torch.float32)
            ref.check(y, *ref.linear(*c))
