"""The workspace of nvfp4_linear against what its scale packing writes, on the
CPU: blocks of 128 rows x 256 of K, 2048 bytes each, two per 256 rows of A, and for B one
per tile of 128 columns or two per tile of 240, whichever width the call takes."""
import ctypes
import random

import pytest


@pytest.fixture(scope="module")
def bytes_of():
    from adaptive_block_scaled_b200 import build
    lib = ctypes.CDLL(build.build())
    f = lib.nvfp4_linear_workspace_bytes
    f.argtypes, f.restype = [ctypes.c_int64] * 3, ctypes.c_size_t
    return f


def ceil(a, b):
    return -(-a // b)


def packed(M, N, K, width, blocks):
    return (ceil(M, 256) * 2 + ceil(N, width) * blocks) * ceil(K, 256) * 2048


def test_it_holds_both_tile_widths(bytes_of):
    rng = random.Random(3)
    sizes = [(rng.randrange(65, 9000), rng.randrange(1, 9000), 32 * rng.randrange(1, 200))
             for _ in range(3000)]
    sizes += [(1 << 22, n, 32) for n in range(1, 1500)] + [(65, 1 << 22, 1 << 20)]
    used = 0
    for M, N, K in sizes:
        have = bytes_of(M, N, K)
        if have:
            used += 1
            assert have >= packed(M, N, K, 128, 1), (M, N, K)
            assert have >= packed(M, N, K, 240, 2), (M, N, K)
    assert used > 2000
