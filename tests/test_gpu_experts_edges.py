"""The experts' layers write their experts' rows and nothing else, and one expert with nearly all rows is as right as any.

The matrices lie in buffers of NaN (test_gpu_linear.matrix), so every element outside the rows of the experts, the rows'
padding and what lies before and behind included, has to be NaN afterwards. Tolerances are those of test_gpu_experts.py."""

import math

import pytest
import torch

import ring_all_reduce_ddp_amd as rar
from test_gpu_experts import FORMS, LAYOUTS, SHAPES, groups, offsets_of
from test_gpu_linear import U, act64, close, gen, matrix, product64, slope64

pytestmark = pytest.mark.gpu


def only_these_written(t, rows):
    """Of the buffer that matrix t lies in, the first `rows` rows of t are numbers and all else is NaN."""
    base = t._base
    assert not bool(torch.isnan(t[:rows].float()).any())
    return int(torch.isnan(base.float()).sum()) == base.numel() - rows * t.shape[1]


def case(counts, behind, n, k, dtype, pad, shift, act="silu"):
    g = gen(11)
    e, rows = len(counts), sum(counts)
    t = rows + behind
    off = offsets_of(counts)
    empty = lambda cols: matrix(g, t, cols, dtype, pad, shift=shift).fill_(math.nan)  # noqa: E731
    x, dz = matrix(g, t, k, dtype, pad, shift=shift), matrix(g, t, n, dtype, pad, shift=shift)
    w = matrix(g, e * n, k, dtype, pad, std=1 / math.sqrt(k), shift=shift).unflatten(0, (e, n))
    zk = matrix(g, t, k, dtype, pad, std=2.0, shift=shift)
    y, z, dx = empty(n), empty(n), empty(k)
    rar.experts_forward(x, w, off, act=act, out=y, z=z)
    rar.experts_backward_input(dz, w, off, act=act, z=zk, out=dx)
    assert only_these_written(y, rows) and only_these_written(z, rows) and only_these_written(dx, rows)
    return x, dz, w, zk, y, z, dx


@pytest.mark.parametrize("layout", LAYOUTS, ids=["dense", "aligned rows", "odd rows"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_nothing_else_is_written(i, dtype, layout):
    counts, behind, n, k = SHAPES[i]
    case(counts, behind + 2, n, k, dtype, *layout)


@pytest.mark.parametrize("direction, dtype, direct, size, form", [f for f in FORMS if f[0] < 2], ids=str)
def test_nothing_else_is_written_in_any_form(direction, dtype, direct, size, form):
    t, e, n, k = size
    cut = sorted(torch.randint(0, t - 2, (e - 1,), generator=torch.Generator().manual_seed(t)).tolist())
    counts = [b - a for a, b in zip([0] + cut, cut + [t - 3])]
    case(counts, 3, n, k, dtype, *((8, 0) if direct else (3, 1)))


# most rows with one expert of many: tiles of 32 rows, as for experts of a few rows each, and parts of sums
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n, k, pad, shift", [(264, 520, 0, 0), (261, 523, 3, 1), (40, 1032, 8, 0)])
@pytest.mark.parametrize("busy", [0, 17, 63])
def test_one_expert_has_nearly_all_rows(busy, n, k, pad, shift, dtype):
    counts = [i % 3 for i in range(64)]
    counts[busy] = 1900
    t, act = sum(counts) + 2, "gelu_tanh"
    for direction in (rar.LINEAR_FORWARD, rar.LINEAR_BACKWARD_INPUT):
        assert rar.experts_tiling(direction, t, 64, n, k, dtype, pad != 3)[0] == 32
    x, dz, w, zk, y, z, dx = case(counts, 2, n, k, dtype, pad, shift, act)
    for i, rows in groups(counts):
        want, _, tol = product64(x[rows], w[i].t())
        close(z[rows], want, tol, dtype, f"z of expert {i}")
        close(y[rows], act64(want, act), 1.13 * tol + 8 * U * want.abs(), dtype, f"y of expert {i}")
        want, _, tol = product64(dz[rows], w[i])
        s = slope64(zk[rows].double(), act)
        close(dx[rows], want * s, tol * (s.abs() + 48 * U) + want.abs() * 48 * U + U * (want * s).abs(), dtype, f"dx of expert {i}")
    dw = torch.full((64, n, k), math.nan, device="cuda")
    rar.experts_backward_weight(dz, x, offsets_of(counts), dw)
    for i, rows in groups(counts):
        want, _, tol = product64(dz[rows].t(), x[rows])
        close(dw[i], want, tol, "fp32", f"dw of expert {i}")
