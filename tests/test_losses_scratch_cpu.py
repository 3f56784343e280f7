"""What the losses of an output layer need as scratch: the bounds that include/ddp_train.h gives."""

import pytest

rar = pytest.importorskip("ring_all_reduce_ddp_amd")

TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]
SIZES = [(1, 1, 1), (7, 1000, 33), (64, 1009, 96), (100, 1 << 20, 64), (1037, 32003, 1001), (4096, 64000, 2048), (8192, 128000, 4096),
         (40000, 9003, 24), (65536, 32000, 1024), (131072, 300, 512), (1 << 20, 4096, 128), (1 << 20, 100, 4096), (1 << 20, 300000, 1)]


def rounded(n, to=256):
    return -(-n // to) * to


@pytest.mark.parametrize("dtype, grads", TYPES)
@pytest.mark.parametrize("m, v, k", SIZES)
@pytest.mark.parametrize("top", [0, 70])
def test_bounds(m, v, k, dtype, grads, top):
    eb = 2 if dtype == "bf16" else 4
    rows = rounded(m * rounded(k, 8) * eb) + 4 * m + 1024
    copy = max(1 << 27, 4096 * rounded(k, 8) * 2) if dtype == "bf16" and k % 8 else 0
    tiles = -(-v // (32 if m <= 32 else 64))
    entries = m * (8 * top + 8 + 2 * (tiles + 1)) + 2048 if top else 0

    def need(direction):
        if top:
            return rar.distill_workspace(direction, m, v, k, top, dtype, grads)
        return rar.cross_entropy_workspace(direction, m, v, k, dtype, grads)

    assert need(rar.LOSS_FORWARD) <= rows + copy + entries + 8 * m * tiles + 4 * m * max(top, 1) + 1024
    if m > 32768:
        values = max(1 << 27, 1024 * m)
    elif (dtype, grads) == ("bf16", "fp32"):
        values = max(1 << 27, 4096 * m)
    else:
        values = max(1 << 25, 4096 * m)
    dz = 4 * (min(values, m * rounded(v, 8)) + 256 * m)   # a piece is whole 256 columns
    assert need(rar.LOSS_BACKWARD) <= rows + copy + entries + dz + 4 * m * k + (1 << 28) + 4096


def test_many_rows_take_little_room_each():
    """2^20 rows: beside 512 bytes of x (256 of bf16) and as much again of dx in fp32, 4 KiB a row of dz."""
    for dtype, grads in TYPES:
        assert rar.cross_entropy_workspace(rar.LOSS_BACKWARD, 1 << 20, 4096, 128, dtype, grads) < (4096 + 1024 + 256) << 20


def test_the_statistics_are_those_of_the_tiles():
    """8192 rows of 128000 columns go in tiles of 256: 8 bytes a row for each, beside 64 MiB of rows."""
    assert rar.loss_tiling(rar.LOSS_Z, 8192, 128000, 4096, "bf16")[1] == 256
    assert rar.loss_tiling(rar.LOSS_Z, 8192, 128000, 4096, "bf16", direct=False)[1] == 128
    assert rar.cross_entropy_workspace(rar.LOSS_FORWARD, 8192, 128000, 4096, "bf16") < (64 << 20) + 8 * 8192 * 1000 + (1 << 20)
