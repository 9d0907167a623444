"""Which tile the products' host rule gives a size, and that product_cases.py has
cases for every one that the rule gives any size."""

import os
import random

import pytest

import moe_grouped_precision_amd as w4a8
from product_cases import CASES


@pytest.fixture(scope="module")
def tile():
    if not os.path.exists(w4a8.lib_path()):
        pytest.fail("libw4a8.so is not built (python -m moe_grouped_precision_amd.build)")
    f = w4a8.load(require_device=False).w4a8_grouped_gemm_tile
    return lambda *a: divmod(f(*a), 1 << 16)


@pytest.mark.parametrize("product,counts,N,K,want", CASES)
def test_a_case_has_its_tile(tile, product, counts, N, K, want):
    assert tile(product, sum(counts), len(counts), N, K) == want


def test_every_tile_has_a_case(tile):
    rng = random.Random(1)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
    found = set()
    for _ in range(60000):
        product = rng.randrange(4)
        N, K = log(32, 16384) // 32 * 32, log(128, 16384) // 128 * 128
        if product < 3 and rng.random() < 0.5:
            N, K = N + rng.randrange(16), K + rng.randrange(16)
        found.add((product, tile(product, log(1, 1 << 20), log(1, 512), N, K)))
    assert found == {(c[0], c[4]) for c in CASES}


def test_only_small_numbers_of_tiles_are_sliced(tile):
    """A size with a workspace for parts of its sum has a tile whose kernel writes them."""
    need = w4a8.load(require_device=False).w4a8_grouped_gemm_workspace_bytes
    rng = random.Random(2)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
    found = set()
    for _ in range(200000):
        product = rng.randrange(4)
        N, K = log(32, 32768) // 32 * 32, log(128, 32768) // 128 * 128
        if product < 3 and rng.random() < 0.5:
            N, K = N + rng.randrange(16), K + rng.randrange(16)
        a = (product, log(1, 1 << 18), log(1, 512), N, K)
        if need(*a):
            found.add((product, tile(*a)))
    assert found == {(0, (64, 128)), (0, (128, 128)), (1, (128, 256)), (1, (128, 128)), (2, (256, 256)), (2, (128, 128)),
                     (3, (64, 128)), (3, (128, 128))}


def test_refused_sizes_have_none(tile):
    for bad in ((4, 9, 1, 64, 128), (-1, 9, 1, 64, 128), (0, 0, 1, 64, 128), (0, -1, 1, 64, 128), (0, 9, 0, 64, 128),
                (0, 9, 2049, 64, 128), (0, 9, 1, 0, 128), (0, 9, 1, 64, 0), (3, 9, 1, 48, 128), (3, 9, 1, 64, 64)):
        assert tile(*bad) == (0, 0)
