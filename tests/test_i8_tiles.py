"""What the library says that a product in the 8-bit form runs as (no GPU)."""
import pytest

import error_bounded_lossy_amd as ec

F = 1 << 20  # a pointer that is never dereferenced
F32, BF16 = 0, 2


@pytest.fixture(scope="module")
def L():
    return ec.lib()


def test_tiles_of_products(L):
    tile = L.ec_i8_product_tile
    assert [tile(r, 8192, 8192, BF16, 0) for r in (1, 16, 17, 64, 512, 8192)] == [16, 16, 64, 64, 128, 256]
    assert [tile(r, 2048, 4096, BF16, 64) for r in (1, 16, 128, 32768)] == [64, 64, 64, 256]
    # outputs of a short contraction are small tiles in fp32
    assert tile(4900, 2500, 1024, BF16, 0) == 256 and tile(4900, 2500, 1024, F32, 0) == 128


# What a product refuses has no tile and no rows that go first.
@pytest.mark.parametrize("rows,cols,depth,kind,experts", [
    (0, 64, 128, BF16, 0), (64, 0, 128, BF16, 0), (64, 64, 0, BF16, 0), (64, 64, 100, BF16, 0), (64, 64, 64, BF16, 2), (64, 64, 128, 3, 0),
    (64, 64, 131072, BF16, 0), (64, 64, 131072, BF16, 2), (1 << 31, 64, 128, BF16, 0), (64, 1 << 31, 128, BF16, 0), (8, 1 << 31, 128, BF16, 0),
    (64, 64, 128, BF16, 1025), (4100, 4096, 131072, BF16, 0), (4100, 4096, 4095, BF16, 0), ((1 << 64) - 1, 64, 128, BF16, 0)])
def test_no_tile_for_what_is_no_product(L, rows, cols, depth, kind, experts):
    assert L.ec_i8_product_tile(rows, cols, depth, kind, experts) == 0
    assert experts or L.ec_i8_product_rows_first(rows, cols, depth, kind) == 0
    if experts:
        assert L.ec_i8_product_experts(F, F, rows, F, F, cols, depth, F, experts, F, kind, None) != ec.EC_OK
    elif rows:
        assert L.ec_i8_product(F, F, rows, F, F, cols, depth, F, kind, None) != ec.EC_OK


def test_rows_that_go_first(L):
    first, tile = L.ec_i8_product_rows_first, L.ec_i8_product_tile
    assert first(4100, 4096, 4096, BF16) == 4096 and tile(4096, 4096, 4096, BF16, 0) == 256
    assert first(2200, 8190, 8064, BF16) == 2048 and tile(152, 8190, 8064, BF16, 0) == 64
    # whole tiles, none, and rows that fit the last round
    assert first(4096, 4096, 4096, BF16) == first(255, 57344, 8192, BF16) == first(4351, 4100, 2048, F32) == 0
