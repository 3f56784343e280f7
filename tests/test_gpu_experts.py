"""The experts' layers (include/ddp_train.h) against 64-bit products of each
expert's rows. Tolerances are those of the linear layer's tests: the products
run through the same sums and outputs."""

import math

import pytest
import torch

import ring_all_reduce_ddp_amd as rar
from test_gpu_linear import ACTS, DT, U, act64, close, gen, matrix, product64, slope64, untouched

pytestmark = pytest.mark.gpu

# rows of each expert, rows behind them, N, K: one row, empty experts at either
# end and between, more experts than rows and than a wave, tiles' edges, a
# long expert beside short ones
SHAPES = [([1], 0, 1, 1), ([0, 3, 0], 2, 7, 5), ([5, 1, 64, 65, 0, 63], 3, 130, 72), ([0] * 40 + [2, 0, 1] + [0] * 50 + [7], 1, 64, 96),
          ([129, 128, 127], 0, 257, 264), ([1] * 130, 0, 72, 40), ([700, 3, 40, 257], 11, 120, 200), ([33, 0, 31], 5, 1032, 640),
          ([0, 0], 4, 16, 24), ([2000, 500], 0, 24, 136)]
LAYOUTS = [(0, 0), (8, 0), (3, 1)]


def offsets_of(counts, first=0):
    return (torch.tensor([0] + list(counts)).cumsum(0) + first).cuda()


def groups(counts, first=0):
    at = first
    for e, n in enumerate(counts):
        yield e, slice(at, at + n)
        at += n


def behind_untouched(t, counts):
    return bool(torch.isnan(t[sum(counts):].float()).all())


def forward_case(counts, behind, n, k, dtype, act, bias, keep, pad, shift, seed=1):
    g = gen(seed)
    e, t = len(counts), sum(counts) + behind
    x = matrix(g, t, k, dtype, pad, shift=shift)
    x[sum(counts):] = math.nan   # rows of nobody
    w = matrix(g, e * n, k, dtype, pad, std=1 / math.sqrt(k), shift=shift).unflatten(0, (e, n))
    b = matrix(g, e, n, dtype) if bias else None
    b = None if b is None else b.contiguous()
    out, z = matrix(g, t, n, dtype, pad, shift=shift), matrix(g, t, n, dtype, pad) if keep else None
    out.fill_(math.nan)
    if keep:
        z.fill_(math.nan)
    rar.experts_forward(x, w, offsets_of(counts), bias=b, act=act, out=out, z=z)
    for i, rows in groups(counts):
        want, _, tol = product64(x[rows], w[i].t())
        if bias:
            want = want + b[i].double()
            tol = tol + U * want.abs()
        if keep:
            close(z[rows], want, tol, dtype, f"z of expert {i}")
        close(out[rows], act64(want, act), 1.13 * tol + 8 * U * want.abs(), dtype, f"y of expert {i}")
    assert behind_untouched(out, counts) and (not keep or behind_untouched(z, counts))


@pytest.mark.parametrize("layout", LAYOUTS, ids=["dense", "aligned rows", "odd rows"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward(i, dtype, layout):
    forward_case(*SHAPES[i], dtype, ACTS[i % 5], i % 2 == 0, i % 3 != 1, *layout)


def input_case(counts, behind, n, k, dtype, act, pad, shift, seed=2):
    g = gen(seed)
    e, t = len(counts), sum(counts) + behind
    dz = matrix(g, t, n, dtype, pad, shift=shift)
    dz[sum(counts):] = math.nan
    w = matrix(g, e * n, k, dtype, pad, std=1 / math.sqrt(n), shift=shift).unflatten(0, (e, n))
    z = matrix(g, t, k, dtype, pad, std=2.0) if act != "none" else None
    out = matrix(g, t, k, dtype, pad, shift=shift)
    out.fill_(math.nan)
    rar.experts_backward_input(dz, w, offsets_of(counts), act=act, z=z, out=out)
    for i, rows in groups(counts):
        want, _, tol = product64(dz[rows], w[i])
        if z is not None:
            s = slope64(z[rows].double(), act)
            tol = tol * (s.abs() + 48 * U) + want.abs() * 48 * U
            want = want * s
        close(out[rows], want, tol + U * want.abs(), dtype, f"dx of expert {i}")
    assert behind_untouched(out, counts)


@pytest.mark.parametrize("layout", LAYOUTS, ids=["dense", "aligned rows", "odd rows"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward_input(i, dtype, layout):
    input_case(*SHAPES[i], dtype, ACTS[(i + 2) % 5], *layout)


def weight_case(counts, behind, n, k, dtype, grads, accumulate, bias, pad, shift, seed=3):
    g = gen(seed)
    e, t = len(counts), sum(counts) + behind
    dz, x = matrix(g, t, n, dtype, pad, shift=shift), matrix(g, t, k, dtype, pad, shift=shift)
    dz[sum(counts):] = math.nan
    x[sum(counts):] = math.nan
    dw = matrix(g, e * n, k, grads, pad, shift=shift)
    db = matrix(g, e, n, grads).contiguous() if bias else None
    old = dw.double().unflatten(0, (e, n)), None if db is None else db.double()
    rar.experts_backward_weight(dz, x, offsets_of(counts), dw.unflatten(0, (e, n)), db, accumulate=accumulate)
    for i, rows in groups(counts):
        want, _, tol = product64(dz[rows].t(), x[rows])
        if accumulate:
            want = want + old[0][i]
            tol = tol + U * want.abs()
        close(dw.unflatten(0, (e, n))[i], want, tol, grads, f"dw of expert {i}")
        if bias:
            want = dz[rows].double().sum(0)
            tol = 2 * (len(dz[rows]) + 2) * U * dz[rows].double().abs().sum(0)
            if accumulate:
                want = want + old[1][i]
                tol = tol + U * want.abs()
            close(db[i], want, tol, grads, f"db of expert {i}")
    assert untouched(dw)


@pytest.mark.parametrize("layout", LAYOUTS, ids=["dense", "aligned rows", "odd rows"])
@pytest.mark.parametrize("types", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")], ids=str)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward_weight(i, types, layout):
    weight_case(*SHAPES[i], *types, i % 2 == 0, i % 3 != 1, *layout)


# enough 256 x 256 tiles for the widest form, with ragged groups
WIDE = [3000, 1, 0, 2500, 2600, 300]


@pytest.mark.parametrize("n, k", [(3600, 136), (136, 3592)])
def test_wide_tiles(n, k):
    forward_case(WIDE, 9, n, k, "bf16", "silu", True, True, 8, 0)
    input_case(WIDE, 9, n, k, "bf16", "silu", 8, 0)
    weight_case(WIDE, 9, n, k, "bf16", "fp32", True, True, 8, 0)
    weight_case(WIDE, 9, n, k, "bf16", "bf16", False, False, 0, 0)


# direction, dtype, whether rows are whole chunks, (T, E, N, K), and the tiles that these give: every form of each product
FORMS = [
    (0, "bf16", False, (5023, 16, 520, 40), (128, 128, 1)), (0, "bf16", False, (3707, 16, 72, 2056), (128, 128, 7)),
    (0, "bf16", False, (60, 8, 264, 2056), (32, 128, 9)), (0, "bf16", False, (300, 16, 1032, 520), (32, 128, 1)), (0, "bf16", False, (19, 2, 40, 2056), (32, 32, 0)),
    (0, "bf16", False, (70, 2, 40, 1032), (64, 64, 0)), (0, "bf16", True, (6392, 8, 264, 40), (128, 128, 1)),
    (0, "bf16", True, (2269, 16, 72, 2056), (128, 128, 7)), (0, "bf16", True, (900, 8, 4104, 40), (128, 256, 1)),
    (0, "bf16", True, (3001, 16, 2056, 40), (256, 256, 1)), (0, "bf16", True, (300, 16, 40, 2056), (32, 128, 0)),
    (0, "bf16", True, (19, 2, 40, 2056), (32, 32, 0)), (0, "bf16", True, (70, 2, 40, 2056), (64, 64, 0)),
    (0, "fp32", False, (5023, 16, 520, 40), (128, 128, 1)), (0, "fp32", False, (4104, 2, 72, 1032), (128, 128, 7)),
    (0, "fp32", False, (60, 8, 264, 1032), (32, 128, 9)), (0, "fp32", False, (300, 16, 1032, 520), (32, 128, 1)), (0, "fp32", True, (5023, 16, 520, 40), (128, 128, 1)),
    (0, "fp32", True, (3707, 16, 72, 2056), (128, 128, 7)), (0, "fp32", True, (300, 16, 40, 1032), (32, 128, 0)),
    (0, "fp32", True, (19, 2, 40, 1032), (32, 32, 0)),
    (1, "bf16", False, (5269, 8, 8, 520), (128, 128, 1)), (1, "bf16", False, (3670, 16, 2056, 72), (128, 128, 7)),
    (1, "bf16", False, (19, 2, 1032, 40), (32, 128, 0)), (1, "bf16", False, (70, 2, 1032, 40), (64, 64, 0)),
    (1, "bf16", True, (6224, 16, 8, 264), (128, 128, 1)), (1, "bf16", True, (2253, 16, 2056, 72), (128, 128, 7)),
    (1, "bf16", True, (900, 16, 8, 2056), (128, 256, 1)), (1, "bf16", True, (900, 8, 4104, 1032), (128, 256, 0)),
    (1, "bf16", True, (2996, 16, 8, 2056), (256, 256, 1)), (1, "bf16", True, (6315, 8, 4104, 520), (256, 256, 3)),
    (1, "bf16", True, (19, 2, 2056, 40), (32, 128, 0)), (1, "bf16", True, (70, 2, 2056, 40), (64, 64, 0)),
    (1, "fp32", False, (5269, 8, 8, 520), (128, 128, 1)), (1, "fp32", False, (3905, 8, 1032, 72), (128, 128, 7)),
    (1, "fp32", True, (5269, 8, 8, 520), (128, 128, 1)), (1, "fp32", True, (1625, 2, 4104, 72), (128, 128, 19)),
    (1, "fp32", True, (19, 2, 1032, 40), (32, 128, 0)),
    (2, "bf16", False, (80, 5, 264, 2056), (128, 128, 1)), (2, "bf16", False, (3095, 2, 2056, 72), (128, 128, 7)),
    (2, "bf16", False, (975, 1, 8, 40), (64, 64, 8)), (2, "bf16", True, (80, 16, 1032, 72), (128, 128, 1)),
    (2, "bf16", True, (4927, 2, 72, 1032), (128, 128, 10)), (2, "bf16", True, (4365, 8, 4104, 136), (256, 256, 1)),
    (2, "bf16", True, (5589, 5, 4104, 136), (256, 256, 3)), (2, "bf16", True, (1412, 1, 8, 40), (64, 64, 6)),
    (2, "fp32", False, (80, 5, 264, 2056), (128, 128, 1)), (2, "fp32", False, (1172, 2, 2056, 72), (128, 128, 7)),
    (2, "fp32", True, (80, 5, 264, 2056), (128, 128, 1)), (2, "fp32", True, (2486, 2, 72, 2056), (128, 128, 7)),
    (2, "fp32", True, (570, 1, 8, 40), (64, 64, 6)),
]


@pytest.mark.parametrize("direction, dtype, direct, size, form", FORMS, ids=str)
def test_every_form(direction, dtype, direct, size, form):
    """form: rows and columns of the tiles, and the parts (0: some number over 1 or 1)."""
    t, e, n, k = size
    got = rar.experts_tiling(direction, t, e, n, k, dtype, direct)
    assert got[:2] == form[:2] and form[2] in (0, got[2]), got
    cut = sorted(torch.randint(0, t + 1, (e - 1,), generator=torch.Generator().manual_seed(t)).tolist())
    counts = [b - a for a, b in zip([0] + cut, cut + [t])]
    layout = (8, 0) if direct else (3, 1)
    if direction == 0:
        forward_case(counts, 0, n, k, dtype, "silu", True, True, *layout)
    elif direction == 1:
        input_case(counts, 0, n, k, dtype, "gelu_tanh", *layout)
    else:
        weight_case(counts, 0, n, k, dtype, "fp32", True, True, *layout)


@pytest.mark.parametrize("bounds", [[-5, 20, 7, 30, 90], [40, 30, 50, 50, 60], [60, 60, 60, 60, 60], [0, 1 << 40, 0, 3, 5],
                                    [-(1 << 60), -3, -2, -1, 0], [10, 20, 30, 40, 50]], ids=str)
def test_bounds_that_do_not_ascend(bounds):
    """Each counts as the largest one up to it within [0, T]: rows outside stay, and no row has two experts."""
    t, e, n, k = 60, 4, 40, 24
    g = gen(4)
    x, w = matrix(g, t, k, "fp32"), matrix(g, e * n, k, "fp32").unflatten(0, (e, n))
    b, seen = [], 0
    for v in bounds:
        seen = max(seen, min(max(v, 0), t))
        b.append(seen)
    out = torch.full((t, n), math.nan, device="cuda")
    off = torch.tensor(bounds, device="cuda")
    rar.experts_forward(x, w, off, out=out)
    dw = torch.full((e, n, k), math.nan, device="cuda")
    db = torch.full((e, n), math.nan, device="cuda")
    rar.experts_backward_weight(out.nan_to_num(), x, off, dw, db)
    for i in range(e):
        rows = slice(b[i], b[i + 1])
        want, _, tol = product64(x[rows], w[i].t())
        close(out[rows], want, tol, "fp32", f"expert {i}")
        want, _, tol = product64(out[rows].t(), x[rows])
        close(dw[i], want, tol, "fp32", f"dw of expert {i}")
    assert bool(torch.isnan(out[:b[0]]).all()) and bool(torch.isnan(out[b[-1]:]).all())


def test_more_experts_than_one_launch_holds():
    """65536 experts of 65 column tiles each: more than 2^22 blocks, for 12 rows."""
    e, n, k = 65536, 65 * 128, 8
    g = gen(8)
    w = torch.empty(e, n, k, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    of = torch.tensor([0, 0, 1, 77, 4095, 30000, 30000, 30000, 50000, 65534, 65535, 65535], device="cuda")
    x = matrix(g, len(of), k, "bf16")
    off = torch.searchsorted(of, torch.arange(e + 1, device="cuda"))
    y = rar.experts_forward(x, w, off)
    for i, o in enumerate(of.tolist()):
        want, _, tol = product64(x[i:i + 1], w[o].t())
        close(y[i:i + 1], want, tol, "bf16", f"row {i}")


def test_no_rows():
    w = torch.ones(3, 5, 8, device="cuda")
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    x, dz = torch.empty(0, 8, device="cuda"), torch.empty(0, 5, device="cuda")
    assert rar.experts_forward(x, w, off).shape == (0, 5)
    assert rar.experts_backward_input(dz, w, off).shape == (0, 8)
    dw, db = torch.ones(3, 5, 8, device="cuda"), torch.ones(3, 5, device="cuda")
    rar.experts_backward_weight(dz, x, off, dw, db, accumulate=True)
    assert bool((dw == 1).all()) and bool((db == 1).all())
    rar.experts_backward_weight(dz, x, off, dw, db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_infinities_and_nan_stay_in_their_rows_and_experts(dtype):
    g = gen(5)
    counts = [100, 70, 30]
    x, dz = matrix(g, 200, 96, dtype), matrix(g, 200, 136, dtype)
    w = matrix(g, 3 * 136, 96, dtype).unflatten(0, (3, 136))
    off = offsets_of(counts)
    x[99, 3], x[100, 5] = math.inf, math.nan
    y = rar.experts_forward(x, w, off).float()
    assert torch.isfinite(y).all(1).tolist() == [i not in (99, 100) for i in range(200)]
    dw = torch.empty(3, 136, 96, device="cuda")
    rar.experts_backward_weight(dz, x, off, dw)
    assert [bool(torch.isfinite(d).all()) for d in dw] == [False, False, True]


def test_one_expert_is_the_linear_layer():
    g = gen(6)
    x, w = matrix(g, 300, 128, "bf16"), matrix(g, 256, 128, "bf16")
    b = matrix(g, 1, 256, "bf16")
    y = rar.experts_forward(x, w[None], offsets_of([300]), bias=b.contiguous(), act="gelu")
    want, z = rar.linear_forward(x, w, bias=b[0].contiguous(), act="gelu", keep=True)
    assert bool(((y.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 1e-5).all())


def test_repeated_calls_streams_and_graphs_give_the_same_bits():
    g = gen(7)
    counts = [70, 0, 129, 41]
    n, k, t, e = 264, 520, 240, 4
    x, dz = matrix(g, t, k, "bf16"), matrix(g, t, n, "bf16")
    w = matrix(g, e * n, k, "bf16").unflatten(0, (e, n))
    z = matrix(g, t, k, "bf16")
    off = offsets_of(counts)
    y, dx = torch.zeros(t, n, device="cuda", dtype=DT["bf16"]), torch.zeros(t, k, device="cuda", dtype=DT["bf16"])
    dw, db = torch.zeros(e, n, k, device="cuda"), torch.zeros(e, n, device="cuda")

    def step(stream=None):
        rar.experts_forward(x, w, off, act="silu", out=y, stream=stream)
        rar.experts_backward_input(dz, w, off, act="silu", z=z, out=dx, stream=stream)
        rar.experts_backward_weight(dz, x, off, dw, db, stream=stream)
        return [a.clone() for a in (y, dx, dw, db)] if stream is None else None

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dw, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shift in (0, 3, -2, 0):   # bounds are read at the replay
        moved = offsets_of([70 + shift, 0, 129 - shift, 41])
        off.copy_(moved)
        want = step()
        for a in (y, dx, dw, db):
            a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dw, db))), shift


@pytest.mark.parametrize("rows", [3, 700])
def test_what_a_workspace_held_reaches_nothing(rows):
    g = gen(8)
    counts, n, k = [rows, 0, 1], 264, 1032
    t, e = rows + 1 + 2, 3
    x, w, dz = matrix(g, t, k, "bf16"), matrix(g, e * n, k, "bf16", std=1 / math.sqrt(k)).unflatten(0, (e, n)), matrix(g, t, n, "bf16")
    x[t - 2:], dz[t - 2:] = math.nan, math.nan
    off = offsets_of(counts)

    def scratch(direction):
        return torch.full((rar.experts_workspace(direction, t, e, n, k, DT["bf16"]),), 255, dtype=torch.uint8, device="cuda")

    y, dx = (torch.full((t, m), math.nan, device="cuda", dtype=DT["bf16"]) for m in (n, k))
    dw, db = torch.full((e, n, k), math.nan, device="cuda"), torch.full((e, n), math.nan, device="cuda")
    rar.experts_forward(x, w, off, out=y, workspace=scratch(rar.LINEAR_FORWARD))
    rar.experts_backward_input(dz, w, off, out=dx, workspace=scratch(rar.LINEAR_BACKWARD_INPUT))
    rar.experts_backward_weight(dz, x, off, dw, db, workspace=scratch(rar.LINEAR_BACKWARD_WEIGHT))
    for i, rows_of in groups(counts):
        want, _, tol = product64(x[rows_of], w[i].t())
        close(y[rows_of], want, tol, "bf16", f"y of expert {i}")
        want, _, tol = product64(dz[rows_of], w[i])
        close(dx[rows_of], want, tol, "bf16", f"dx of expert {i}")
        want, _, tol = product64(dz[rows_of].t(), x[rows_of])
        close(dw[i], want, tol, "fp32", f"dw of expert {i}")
        want = dz[rows_of].double().sum(0)
        close(db[i], want, 2 * (counts[i] + 2) * U * dz[rows_of].double().abs().sum(0), "fp32", f"db of expert {i}")
    assert behind_untouched(y, counts) and behind_untouched(dx, counts)


def test_arguments():
    x, w = torch.zeros(6, 8, device="cuda"), torch.zeros(2, 4, 8, device="cuda")
    off = torch.tensor([0, 3, 6], device="cuda")
    dz = torch.zeros(6, 4, device="cuda")
    with pytest.raises(ValueError, match="offsets"):
        rar.experts_forward(x, w, off[:2])
    with pytest.raises(ValueError, match="offsets"):
        rar.experts_forward(x, w, off.int())
    with pytest.raises(ValueError, match="offsets"):
        rar.experts_forward(x, w, off.cpu())
    with pytest.raises(ValueError, match="w must be"):
        rar.experts_forward(x, torch.zeros(2, 4, 7, device="cuda"), off)
    with pytest.raises(ValueError, match="evenly"):
        rar.experts_forward(x, torch.zeros(4, 4, 8, device="cuda")[::2], off)
    with pytest.raises(ValueError, match="bias"):
        rar.experts_forward(x, w, off, bias=torch.zeros(8, device="cuda"))
    with pytest.raises(rar.DDPError, match="overlaps"):
        rar.experts_backward_input(dz, torch.zeros(2, 4, 4, device="cuda"), off, out=dz)
    with pytest.raises(rar.DDPError, match="needs z"):
        rar.experts_backward_input(dz, w, off, act="relu")
    with pytest.raises(rar.DDPError, match="K must"):
        rar.experts_forward(torch.zeros(6, 0, device="cuda"), torch.zeros(2, 4, 0, device="cuda"), off)
    with pytest.raises(rar.DDPError, match="grad_dtype"):
        rar.experts_backward_weight(dz, x, off, torch.zeros(2, 4, 8, device="cuda", dtype=torch.bfloat16))
