"""The adapters' workspace size: it does not decrease in any argument, so that one
workspace, of the largest call's size, serves every smaller call. No GPU needed."""
import random

import pytest

from w8a8_quantized_matmul_b200 import _lib
from w8a8_quantized_matmul_b200 import build as _build


@pytest.fixture(scope="module")
def size():
    _build.build()
    return _lib.load().int8_adapter_add_workspace_size


def test_it_does_not_shrink_as_the_batch_grows(size):
    for K, n, R in ((8192, 48, 16), (8192, 4, 64), (528, 4, 16), (65536, 4096, 128), (4096, 31, 8), (4096, 32, 8), (64, 1, 40)):
        last = 0
        for M in range(1, 1200):
            now = size(M, 4096, K, n, R)
            assert now >= last > -1 and now > 0, (M, K, n, R)
            last = now
        assert size(1 << 22, 4096, K, n, R) >= last


def test_it_does_not_shrink_in_any_argument(size):
    rng = random.Random(5)
    for _ in range(4000):
        big = [rng.choice([rng.randint(1, 1100), rng.randint(1, 1 << 22)]), rng.randint(1, 1 << 22), 16 * rng.randint(1, 4096),
               rng.choice([rng.randint(1, 64), rng.randint(1, 4096)]), 8 * rng.randint(1, 16)]
        small = [rng.randint(1, big[0]), rng.randint(1, big[1]), 16 * rng.randint(1, big[2] // 16), rng.randint(1, big[3]),
                 8 * rng.randint(1, big[4] // 8)]
        for i in range(5):   # one argument at a time, then all
            one = list(big)
            one[i] = small[i]
            assert size(*one) <= size(*big), (one, big)
        assert size(*small) <= size(*big), (small, big)


def test_it_stays_small(size):
    """The tiles' form takes what it needs, the other at most 1 MB and its control words."""
    for M, K, n, R in ((16, 4096, 8, 16), (1024, 8192, 48, 16), (192, 8192, 4, 64), (1025, 8192, 48, 16), (4096, 8192, 6, 64), (20000, 65536, 4096, 128)):
        kinds = min(n + 1, M)
        tiles = M * (4 * R + 8) + 16 * (M // 128 + kinds) + 256 * 6
        assert size(M, 64, K, n, R) <= max(tiles, (1 << 20) + 512)
