"""Which weights of a loss are copied to rows of whole 16 bytes, by the tiles that the products get: where the
copy costs the forward pass more than it saves, small vocabularies and few products, there is none."""

import pytest

rar = pytest.importorskip("ring_all_reduce_ddp_amd")

# sizes whose tiles differ with and without whole chunks
SMALL = [(2050, 5003, 501), (4100, 5003, 501), (2050, 5003, 1001)]
LARGE = [(8000, 32003, 2047), (4100, 12003, 1001), (2050, 32003, 501), (8000, 5003, 135), (4100, 128003, 135)]


def tiles(product, size, direct):
    return rar.loss_tiling(product, *size, "bf16", "bf16", direct)


@pytest.mark.parametrize("size", SMALL, ids=str)
def test_small_vocabularies_are_read_as_they_are(size):
    assert tiles(rar.LOSS_Z, size, True)[:2] == (256, 256) and tiles(rar.LOSS_Z, size, False)[:2] == (128, 128)


@pytest.mark.parametrize("size", LARGE, ids=str)
def test_large_ones_are_copied(size):
    assert tiles(rar.LOSS_Z, size, False) == tiles(rar.LOSS_Z, size, True)


@pytest.mark.parametrize("size", SMALL + LARGE, ids=str)
def test_backward_two_products_read_the_copy(size):
    assert tiles(rar.LOSS_Z_AGAIN, size, False) == tiles(rar.LOSS_Z_AGAIN, size, True)


@pytest.mark.parametrize("m, v, k", [(2047, 128003, 2047), (8000, 32003, 127), (1030, 32003, 1001)])
def test_few_rows_and_short_ones_are_not(m, v, k):
    assert tiles(rar.LOSS_Z, (m, v, k), False)[:2] == (128, 128) != tiles(rar.LOSS_Z, (m, v, k), True)[:2]
