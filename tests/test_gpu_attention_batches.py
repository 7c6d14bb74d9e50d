"""GPU tier: attention over batches of unusual make-up."""
import pytest
import torch

from tests.test_gpu_decoder_ops import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tenant_fine_tune_amd as bd

    return bd


def test_padding_alone_with_groups(bd):
    """No sequences, no arrays of sequences, groups that are still there: zero rows."""
    import ctypes

    from tenant_fine_tune_amd import decoder

    kv = bd.PagedKV.empty(4, 2, 16, 64)
    start, lens, table = i32([0, 3]), i32([40]), i32([[0, 1, 2]])
    b = decoder._Batch(None, None, None, start.data_ptr(), lens.data_ptr(), table.data_ptr(), 5, 0, 0, 1, 3, 0)
    q = torch.ones(5, 8, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.ones_like(q)
    need = bd.lib.bitdelta_attention_workspace(8, kv._ref, ctypes.addressof(b))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    assert bd.lib.bitdelta_attention(q.data_ptr(), 512, 8, 0.1, kv._ref, ctypes.addressof(b), out.data_ptr(),
                                     ws.data_ptr(), need, st) == bd.BD_OK
    assert not out.any()
    out.fill_(1)
    k = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert bd.lib.bitdelta_kv_append(q.data_ptr(), 512, k.data_ptr(), 128, k.data_ptr(), 128, 8, None, 0, 0, kv._ref,
                                     ctypes.addressof(b), out.data_ptr(), st) == bd.BD_OK
    assert not out.any()
