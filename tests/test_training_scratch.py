"""CPU checks of the scratch memory that the training operators ask for."""
import ctypes

import pytest

import adaptive_gradient_summation_gb300 as ags


@pytest.mark.parametrize("n,cols,K", [(65_536, 1024, 16), (1 << 20, 4096, 1), (60_000, 256, 3), (1 << 20, 16, 1)])
def test_table_gradient_asks_for_what_it_uses(n, cols, K):
    """Keys and places twice (16 bytes a token), digit counts (4 bytes a token and 5 KiB a worker),
    two partial rows per chunk of 8, 16 or 32 tokens a warp, as there are columns to sum."""
    offs = (ctypes.c_int64 * (K + 1))(*(n * k // K for k in range(K + 1)))
    got = ags.load_library().adasum_embedding_backward_scratch_bytes(offs, K, 30_522, cols)
    work = n * -(-cols // 256)
    part = 32 if work >= 150_000 else 16 if work >= 50_000 else 8
    chunks = n // (8 * part) + K
    assert got <= 20 * n + 5 * 1024 * K + chunks * (8 * cols + 4) + 9 * 256
    assert got >= 16 * n + chunks * 8 * cols
