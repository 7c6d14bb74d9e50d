"""CPU tier: matrices of so many rows that a launch of a workgroup or a wave a
row would need 2^32 threads, which wraps around without an error and leaves
rows undone, are refused."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def bd():
    import tenant_fine_tune_amd as bd

    return bd


def test_more_rows_than_a_launch_takes_are_refused(bd):
    lib, big = bd.lib, 1 << 40
    for rows in (1 << 24, (1 << 24) + 3, (1 << 31) - 1):
        assert lib.bitdelta_compress(FAKE, FAKE, 0, rows, 8, 0, FAKE, FAKE, FAKE, big, None) == bd.BD_ESHAPE
        assert lib.bitdelta_compress(FAKE, FAKE, 1, rows, 64, 1, FAKE, FAKE, FAKE, big, None) == bd.BD_ESHAPE
        assert lib.bitdelta_reconstruct(FAKE, FAKE, FAKE, 0, rows, 8, FAKE, None) == bd.BD_ESHAPE
        assert lib.bitdelta_similarity_delta(FAKE, FAKE, 0, 14, rows, 8, FAKE, FAKE, FAKE, big, None) == bd.BD_ESHAPE
    # four workgroups a row of 8192 columns
    assert lib.bitdelta_reconstruct(FAKE, FAKE, FAKE, 0, 1 << 22, 8192, FAKE, None) == bd.BD_ESHAPE
    for m in (1, 2, 4, 16):
        assert lib.bitdelta_linear(FAKE, m, FAKE, FAKE, FAKE, 0, 1 << 26, 8, FAKE, FAKE, big, None) == bd.BD_ESHAPE
