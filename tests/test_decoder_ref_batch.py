"""CPU tier: the 64-bit form of attention by sequences is the one by tokens."""
import numpy as np

from tests import decoder_ref as ref
from tests import decoder_ref_batch as ref_batch


def test_by_sequence_is_by_token():
    host = ref.Batch([0, 3, 3, 4, 9], [8, 0, 1, 5], [[4, 2, 0], [0, 0, 0], [1, -1, 0], [9, 3, 5]], 4, 7, [1, 4], [6], [[6, 2]])
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((10, 4, 8)), rng.standard_normal((7, 2, 4, 8)), rng.standard_normal((7, 2, 4, 8))
    for kv_len in ([8, 0, 1, 5], [2, 0, 0, 12]):
        host.kv_len = np.array(kv_len)
        for a, b in zip(ref.attention(q, k, v, host, 0.3), ref_batch.attention(q, k, v, host, 0.3)):
            assert np.allclose(a, b, rtol=1e-12, atol=1e-15)
