"""The linear layer's products (include/ddp_train.h) against 64-bit products
of the same inputs.

Tolerances, with u = 2^-24 (fp32) and b = 2^-8 (bf16), the largest relative
errors of one rounding to nearest, and A = sum |a b| of a sum of K terms:
- a sum in fp32 with any order, and truncation instead of rounding inside the
  matrix instruction: 2 (K + 2) u A;
- an activation's value: 8 u |z| (the exponential's relative error is at most
  2 u times its argument, which the sigmoid's slope takes back), and the error
  of z times a slope of at most 1.13;
- its slope: 48 u (gelu_tanh's 1 - s, whose error u meets z (1.6 + 0.21 z^2) up
  to where s is 1, z = 5.3; the others are smaller);
- bias, residual, add, old gradient: u of the sum each;
- the result's rounding: u or b of it, and half the smallest subnormal.
"""

import math

import pytest
import torch

import ring_all_reduce_ddp_amd as rar

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]

# M, N, K: single elements and rows, odd sizes below and above a tile, sums cut
# into parts, several tiles with edges on each side
SIZES = [(1, 1, 1), (1, 64, 64), (1, 1000, 2049), (1, 4096, 1024), (2, 72, 520), (3, 5, 7), (7, 1023, 264), (8, 256, 4096),
         (9, 130, 1000), (17, 33, 65), (64, 64, 4096), (128, 128, 64), (129, 127, 63), (136, 264, 72), (256, 384, 128),
         (300, 257, 513), (1037, 120, 200), (2, 3, 5001), (640, 648, 1032)]
# enough 256 x 256 tiles for each direction's widest form, with ragged edges
LARGE = [(3592, 3600, 136), (3600, 136, 3592), (136, 3592, 3600)]


def matrix(g, rows, cols, dtype, pad=0, std=1.0, shift=0):
    """rows x cols with `pad` more elements per row and `shift` before the
    first, all of those NaN: nothing outside the matrix may matter."""
    full = torch.full((shift + rows * (cols + pad) + 8,), math.nan, device="cuda").to(DT[dtype])
    t = full[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda") * std)
    return t


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    z = z.clone().requires_grad_(True)
    with torch.enable_grad():
        (s,) = torch.autograd.grad(act64(z, act).sum(), z)
    return s


def product64(a, b):
    """(a b, sum |a b|, and the bound of an fp32 sum) in 64 bits."""
    a, b = a.double(), b.double()
    mag = a.abs() @ b.abs()
    return a @ b, mag, 2 * (a.shape[1] + 2) * U * mag


def close(got, want, tol, dtype, what):
    r = U if dtype == "fp32" else B
    lim = tol + r * (want.abs() + tol) + (2.0 ** -149 if dtype == "fp32" else 2.0 ** -133)
    bad = ~((got.double() - want).abs() <= lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


def untouched(t):
    """The elements around a matrix made by matrix() are still NaN."""
    base = t._base if t._base is not None else t
    inside = t.numel()
    return int(torch.isnan(base.float()).sum()) == base.numel() - inside


def forward_case(m, n, k, dtype, act, bias, residual, keep, pad, shift, seed=1):
    g = gen(seed)
    x = matrix(g, m, k, dtype, pad, shift=shift)
    w = matrix(g, n, k, dtype, pad, std=1 / math.sqrt(k), shift=shift)
    bv = matrix(g, 1, n, dtype)[0] if bias else None
    r = matrix(g, m, n, dtype, pad) if residual else None
    out = matrix(g, m, n, dtype, pad, shift=shift)
    z = matrix(g, m, n, dtype, pad, shift=shift) if keep else None
    rar.linear_forward(x, w, bias=bv, residual=r, act=act, out=out, z=z)
    want, mag, tol = product64(x, w.t())
    if bias:
        want = want + bv.double()
        tol = tol + U * want.abs()
    if keep:
        close(z, want, tol, dtype, "z")
        assert untouched(z)
    y = act64(want, act)
    tol = 1.13 * tol + 8 * U * want.abs()
    if residual:
        y = y + r.double()
        tol = tol + U * y.abs()
    close(out, y, tol, dtype, "y")
    assert untouched(out)


@pytest.mark.parametrize("layout", [(0, 0), (8, 0), (3, 1)], ids=["dense", "aligned rows", "odd rows"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dtype, layout):
    i = SIZES.index(size)
    forward_case(*size, dtype, ACTS[i % 5], i % 2 == 0, i % 3 != 0, i % 4 != 1, *layout)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 5, 40, 300])
def test_forward_activations(rows, dtype, act):
    forward_case(rows, 264, 96, dtype, act, True, True, True, 0, 0)
    forward_case(rows, 264, 96, dtype, act, False, False, False, 0, 0)


def input_case(m, n, k, dtype, act, add, pad, shift, seed=2):
    g = gen(seed)
    dz = matrix(g, m, n, dtype, pad, shift=shift)
    w = matrix(g, n, k, dtype, pad, std=1 / math.sqrt(n), shift=shift)
    z = matrix(g, m, k, dtype, pad, std=2.0) if act != "none" else None
    a = matrix(g, m, k, dtype, pad) if add else None
    out = matrix(g, m, k, dtype, pad, shift=shift)
    rar.linear_backward_input(dz, w, act=act, z=z, add=a, out=out)
    want, mag, tol = product64(dz, w)
    if z is not None:
        s = slope64(z.double(), act)
        tol = tol * (s.abs() + 48 * U) + want.abs() * 48 * U
        want = want * s
    if add:
        want = want + a.double()
        tol = tol + U * want.abs()
    close(out, want, tol + U * want.abs(), dtype, "dx")
    assert untouched(out)


@pytest.mark.parametrize("layout", [(0, 0), (8, 0), (3, 1)], ids=["dense", "aligned rows", "odd rows"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward_input(size, dtype, layout):
    i = SIZES.index(size)
    input_case(*size, dtype, ACTS[(i + 2) % 5], i % 3 == 0, *layout)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_backward_input_activations(dtype, act):
    input_case(70, 96, 264, dtype, act, True, 0, 0)
    input_case(1, 96, 264, dtype, act, False, 0, 0)


def weight_case(m, n, k, dtype, grads, accumulate, bias, pad, shift, seed=3):
    g = gen(seed)
    dz = matrix(g, m, n, dtype, pad, shift=shift)
    x = matrix(g, m, k, dtype, pad, shift=shift)
    dw = matrix(g, n, k, grads, pad, shift=shift)
    db = matrix(g, 1, n, grads, 0, shift=shift)[0] if bias else None
    old = dw.double(), None if db is None else db.double()
    rar.linear_backward_weight(dz, x, dw, db, accumulate=accumulate)
    want, mag, tol = product64(dz.t(), x)
    if accumulate:
        want = want + old[0]
        tol = tol + U * want.abs()
    close(dw, want, tol, grads, "dw")
    assert untouched(dw)
    if bias:
        want = dz.double().sum(0)
        tol = 2 * (m + 2) * U * dz.double().abs().sum(0)
        if accumulate:
            want = want + old[1]
            tol = tol + U * want.abs()
        close(db, want, tol, grads, "db")


@pytest.mark.parametrize("layout", [(0, 0), (8, 0), (3, 1)], ids=["dense", "aligned rows", "odd rows"])
@pytest.mark.parametrize("types", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward_weight(size, types, layout):
    i = SIZES.index(size)
    weight_case(*size, *types, i % 2 == 0, i % 3 != 1, *layout)


@pytest.mark.parametrize("size", LARGE, ids=str)
@pytest.mark.parametrize("what", ["forward", "input", "weight"])
def test_wide_tiles(what, size):
    m, n, k = size
    if what == "forward":
        forward_case(m, n, k, "bf16", "gelu_tanh", True, True, True, 8, 0)
    elif what == "input":
        input_case(m, n, k, "bf16", "silu", True, 8, 0)
    else:
        weight_case(m, n, k, "bf16", "fp32", True, True, 8, 0)
        weight_case(m, n, k, "bf16", "bf16", False, False, 0, 0)


def test_zero_sizes():
    e = lambda r, c: torch.empty(r, c, device="cuda")  # noqa: E731
    assert rar.linear_forward(e(0, 5), e(3, 5)).shape == (0, 3)
    assert rar.linear_forward(e(4, 5), e(0, 5)).shape == (4, 0)
    bias = torch.arange(-3.0, 3.0, device="cuda")
    y, z = rar.linear_forward(e(2, 0), e(6, 0), bias=bias, act="relu", keep=True)
    assert torch.equal(z, bias.expand(2, 6)) and torch.equal(y, bias.clamp(min=0).expand(2, 6))
    add = torch.randn(3, 4, device="cuda")
    assert torch.equal(rar.linear_backward_input(e(3, 0), e(0, 4), add=add), add)
    dw, db = torch.ones(6, 4, device="cuda"), torch.ones(6, device="cuda")
    rar.linear_backward_weight(e(0, 6), e(0, 4), dw, db, accumulate=True)
    assert bool((dw == 1).all()) and bool((db == 1).all())
    rar.linear_backward_weight(e(0, 6), e(0, 4), dw, db)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    db = torch.zeros(6, device="cuda")
    rar.linear_backward_weight(torch.ones(5, 6, device="cuda"), e(5, 0), e(6, 0), db)
    assert bool((db == 5).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_infinities_and_nan_stay_in_their_rows(dtype):
    g = gen(4)
    x = matrix(g, 200, 96, dtype)
    w = matrix(g, 136, 96, dtype)
    x[7, 3] = math.inf
    x[150, 90] = math.nan
    y = rar.linear_forward(x, w).float()
    ok = torch.isfinite(y).all(1)
    assert ok.tolist() == [i not in (7, 150) for i in range(200)]
    assert bool(torch.isnan(y[150]).all()) and bool(torch.isinf(y[7]).all())


def test_extreme_preactivations():
    """Large |z| saturate: no NaN from an overflowing exponential."""
    z = torch.tensor([[-1e30, -300.0, -90.0, -20.0, 0.0, 20.0, 90.0, 300.0, 1e30]], device="cuda")
    one = torch.ones(1, 1, device="cuda")
    for act in ACTS:
        y = rar.linear_forward(one, z.t().contiguous(), act=act)
        want = z if act == "none" else z.clamp(min=0)
        assert bool(((y - want).abs() <= 1e-6 * want.abs() + 1e-6).all()), (act, y)
        s = rar.act_backward(torch.ones_like(z), z, act)
        want = torch.ones_like(z) if act == "none" else (z > 0).float() + (0.5 * (z == 0) if act != "relu" else 0)
        assert bool(((s - want).abs() <= 1e-6).all()), (act, s)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """Central differences of the forward pass along random directions of x, w
    and the bias. L = sum(c * y) over 6 x 10 outputs of 8 terms: each y is off
    by at most 2 * 10 u A + 8 u |z| < 3e-5 (A and |z| below 20), so the quotient
    by at most 3e-5 * sum|c| / h; the third derivative along a direction whose
    effect on z is D is below 2 |D|^3 (its largest value for these
    activations), which adds h^2 / 3 * sum(|c| |D|^3)."""
    m, n, k, h = 6, 10, 8, 0.03
    g = gen(5)
    x, w = matrix(g, m, k, "fp32"), matrix(g, n, k, "fp32", std=0.3)
    if act == "relu":
        x = x.abs().contiguous()   # z away from relu's corner
        w = w.abs().contiguous()
    b = matrix(g, 1, n, "fp32")[0].contiguous()
    if act == "relu":
        b = b.abs() + 1.0
    c = matrix(g, m, n, "fp32")
    _, z = rar.linear_forward(x, w, bias=b, act=act, keep=True)
    dz = rar.act_backward(c, z, act)
    dx = rar.linear_backward_input(dz, w)
    dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    rar.linear_backward_weight(dz, x, dw, db)
    for name in ("x", "w", "b"):
        p, grad = {"x": (x, dx), "w": (w, dw), "b": (b, db)}[name]
        d = torch.randn(p.shape, generator=g, device="cuda") * (0.3 if act == "relu" else 1.0)
        if act == "relu":
            d = d.clamp(-1, 1)
        at = {"x": x, "w": w, "b": b}

        def loss(t):
            q = {**at, name: (p + t * d).contiguous()}
            return float((c.double() * rar.linear_forward(q["x"], q["w"], bias=q["b"], act=act).double()).sum())

        q = {name: d.double()}
        effect = d.double() @ w.double().t() if name == "x" else x.double() @ d.double().t() if name == "w" else d.double().expand(m, n)
        tol = 3e-5 * float(c.abs().sum()) / h + h * h / 3 * float((c.double().abs() * effect.abs() ** 3).sum())
        assert abs((loss(h) - loss(-h)) / (2 * h) - float((grad.double() * q[name]).sum())) <= tol, name


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("pad", [0, 3])
def test_act_backward(pad, act, dtype):
    g = gen(6)
    dy, z = matrix(g, 37, 129, dtype, pad, shift=1), matrix(g, 37, 129, dtype, pad, std=2.0)
    out = matrix(g, 37, 129, dtype, pad)
    rar.act_backward(dy, z, act, out=out)
    want = dy.double() * slope64(z.double(), act)
    close(out, want, 48 * U * dy.double().abs(), dtype, "dz")
    assert untouched(out)
    rar.act_backward(dy, z, act, out=dy)
    assert torch.equal(dy, out)


def test_in_place_residual_and_add():
    g = gen(7)
    x, w = matrix(g, 300, 128, "bf16"), matrix(g, 256, 128, "bf16")
    r = matrix(g, 300, 256, "bf16")
    want = rar.linear_forward(x, w, residual=r, act="silu")
    rar.linear_forward(x, w, residual=r, act="silu", out=r)
    assert torch.equal(r, want)
    a = matrix(g, 300, 128, "bf16")
    want = rar.linear_backward_input(r, w, add=a)
    rar.linear_backward_input(r, w, add=a, out=a)
    assert torch.equal(a, want)


@pytest.mark.parametrize("size", [(1, 512, 512), (64, 264, 4096), (513, 520, 264)], ids=str)
def test_repeated_calls_give_the_same_bits(size):
    m, n, k = size
    g = gen(8)
    x, w, dz = matrix(g, m, k, "bf16"), matrix(g, n, k, "bf16"), matrix(g, m, n, "bf16")

    def results():
        dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
        rar.linear_backward_weight(dz, x, dw, db)
        return [rar.linear_forward(x, w, act="gelu"), rar.linear_backward_input(dz, w), dw, db]

    first = results()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(results(), first))


def test_on_another_stream_and_in_a_graph():
    g = gen(9)
    m, n, k = 96, 136, 2048   # sums in parts
    x, w, dz = matrix(g, m, k, "bf16"), matrix(g, n, k, "bf16"), matrix(g, m, n, "bf16")
    side = torch.cuda.Stream()
    dw, db = torch.zeros(n, k, device="cuda"), torch.zeros(n, device="cuda")
    y, dx = torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(rar.linear_workspace(d, m, n, k, "bf16") for d in range(3)), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        rar.linear_forward(x, w, act="relu", out=y, workspace=ws, stream=stream)
        rar.linear_backward_input(dz, w, out=dx, workspace=ws, stream=stream)
        rar.linear_backward_weight(dz, x, dw, db, workspace=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, dw, db)]
    for t in (y, dx, dw, db):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, dx, dw, db), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
            step()
    for _ in range(4):
        for t in (y, dx, dw, db):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw, db), want))


def test_gradients_into_an_arena():
    """The weight's and the bias's gradient as views of a gradient arena, over
    two micro-batches, and nothing else of the arena touched."""
    g = gen(10)
    n, k = 33, 70
    plan = rar.ddp_bucket_plan([5, n * k, n, 9], "fp32", world_size=1)
    length, offs = plan.grad_arena()
    arena = torch.full((length,), math.nan, device="cuda")
    dw, db = arena[offs[1]:offs[1] + n * k].view(n, k), arena[offs[2]:offs[2] + n]
    want_w, want_b = 0.0, 0.0
    for i in range(2):
        dz, x = matrix(g, 50, n, "bf16"), matrix(g, 50, k, "bf16")
        rar.linear_backward_weight(dz, x, dw, db, accumulate=i > 0)
        want_w, want_b = want_w + dz.double().t() @ x.double(), want_b + dz.double().sum(0)
    assert bool(((dw - want_w).abs() <= 1e-4).all()) and bool(((db - want_b).abs() <= 1e-4).all())
    assert int(torch.isnan(arena).sum()) == length - n * k - n


def test_refusals():
    f = torch.float32
    x, w, y = (torch.ones(*s, device="cuda") for s in ((8, 16), (4, 16), (8, 4)))
    with pytest.raises(ValueError, match="w must be"):
        rar.linear_forward(x, torch.ones(4, 15, device="cuda"))
    with pytest.raises(ValueError, match="w must be"):
        rar.linear_forward(x, w.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        rar.linear_forward(torch.ones(16, 8, device="cuda").t(), w)
    with pytest.raises(ValueError, match="bias must be"):
        rar.linear_forward(x, w, bias=torch.ones(5, device="cuda"))
    with pytest.raises(ValueError, match="unsupported dtype"):
        rar.linear_forward(x.half(), w.half())
    with pytest.raises(KeyError):
        rar.linear_forward(x, w, act="tanh")
    with pytest.raises(rar.DDPError, match="overlaps"):
        rar.linear_forward(x, w, out=x[:, :4])
    with pytest.raises(rar.DDPError, match="overlaps"):
        rar.linear_forward(x, w, out=y, z=y)
    with pytest.raises(rar.DDPError, match="needs z"):
        rar.linear_backward_input(y, w, act="relu")
    with pytest.raises(rar.DDPError, match="overlaps"):
        rar.linear_backward_input(y, w, z=x, out=x)
    with pytest.raises(rar.DDPError, match="grad_dtype"):
        rar.linear_backward_weight(y, x, torch.ones(4, 16, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(rar.DDPError, match="overlaps"):
        rar.linear_backward_weight(y, x, torch.ones(4, 16, device="cuda"), db=y.view(-1)[:4])
    need = rar.linear_workspace(rar.LINEAR_FORWARD, 64, 64, 8192, "fp32")
    assert need > 0
    a, b = torch.ones(64, 8192, device="cuda"), torch.ones(64, 8192, device="cuda")
    with pytest.raises(rar.DDPError, match="workspace needs"):
        rar.linear_forward(a, b, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    small = torch.ones(8, 16, device="cuda")
    lib = rar.lib
    args = lambda ldx, m=8: (small.data_ptr(), ldx, w.data_ptr(), 16, None, None, 4, y.data_ptr(), 4, None, 4, m, 4, 16, 0, 0, None, 0, None)  # noqa: E731
    assert lib.ddp_linear_forward(*args(15)) == rar.DDP_EINVAL and b"leading dimension" in lib.ddp_last_error()
    assert lib.ddp_linear_forward(*args(1 << 30)) == rar.DDP_EINVAL and b"past the end" in lib.ddp_last_error()
    assert lib.ddp_linear_forward(*args(16, m=-1)) == rar.DDP_EINVAL and b"M, N and K" in lib.ddp_last_error()
    assert f is torch.float32


@pytest.mark.parametrize("size, dtype, layout", [((8201, 5600, 72), "bf16", (0, 0)), ((8201, 5603, 41), "bf16", (3, 1)),
                                                 ((5001, 4600, 40), "fp32", (0, 0))], ids=str)
def test_kept_z_beyond_the_cache(size, dtype, layout):
    """y and z of over two thirds of the Infinity Cache: z's stores pass it."""
    forward_case(*size, dtype, "gelu", True, False, True, *layout)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("m, n, k", [(300, 256, 128), (70, 33, 41), (3, 72, 40)])
def test_column_blocks_of_one_buffer(m, n, k, dtype):
    """Inputs and outputs side by side in one buffer: the results of separate ones, and the inputs stay."""
    g = gen(11)
    x, w, r = matrix(g, m, k, dtype), matrix(g, n, k, dtype), matrix(g, m, n, dtype)
    want, want_z = rar.linear_forward(x, w, residual=r, act="silu", keep=True)
    want_dx = rar.linear_backward_input(r, w, add=x)
    wide = torch.full((m, 3 * n + k), math.nan, device="cuda").to(DT[dtype])
    y, z, r2, x2 = wide.split([n, n, n, k], 1)
    r2.copy_(r)
    x2.copy_(x)
    rar.linear_forward(x2, w, residual=r2, act="silu", out=y, z=z)
    # loads of another alignment may take another cut of the sum
    tol = 4 * (k + 2) * U * (x.double().abs() @ w.double().abs().t())
    close(z, want_z.double(), tol + (B if dtype == "bf16" else U) * want_z.double().abs(), dtype, "z")
    close(y, want.double(), 2 * tol + 2 * (B if dtype == "bf16" else 8 * U) * (want.double().abs() + r.double().abs()), dtype, "y")
    assert torch.equal(x2, x) and torch.equal(r2, r)
    wide = torch.full((m, 2 * k + n), math.nan, device="cuda").to(DT[dtype])
    dx, a, dz = wide.split([k, k, n], 1)
    a.copy_(x)
    dz.copy_(r)
    rar.linear_backward_input(dz, w, add=a, out=dx)
    tol = 4 * (n + 2) * U * (r.double().abs() @ w.double().abs())
    close(dx, want_dx.double(), tol + (B if dtype == "bf16" else U) * (want_dx.double().abs() + x.double().abs()), dtype, "dx")
    assert torch.equal(a, x) and torch.equal(dz, r)


def act_and_bound(z, act):
    """An activation in 64 bits, without sums that cancel for negative z, and
    the most that its fp32 form may be off for exact z. The library's
    erfc is taken as good to 8u (4 ulp), its exponential to 4u.
    - gelu: x = |z| / sqrt 2 is off by 1.3u of itself, which erfc's condition
      number takes up to z^2 + 1 times: q = erfc(x) / 2 to u (1.3 z^2 + 9.3). The
      function is q, or 1 - q with u/2 more, and the product u.
    - gelu_tanh: the exponent w = z (k1 + k3 z^2) is off by 4.5u of itself (two
      constants, square, fma, product), which 1 / (1 + exp(-w)) takes 1 - s
      times; sum and quotient u each.
    - silu: the same without the exponent's errors.
    The smallest subnormal times z comes to that."""
    tiny = 2.0 ** -149 * (z.abs() + 1)
    if act == "gelu":
        y = z * torch.special.erfc(-z * math.sqrt(0.5)) / 2
        q = torch.special.erfc(z.abs() * math.sqrt(0.5)) / 2
        return y, z.abs() * U * (q * (1.3 * z * z + 9.3) + 0.5 * (z > 0)) + U * y.abs() + tiny
    w = z * (math.sqrt(8 / math.pi) * (1 + 0.044715 * z * z)) if act == "gelu_tanh" else z
    y = z * torch.sigmoid(w)
    return y, y.abs() * U * (torch.sigmoid(-w) * (4 + (4.5 * w.abs() if act == "gelu_tanh" else 0)) + 2) * 1.0001 + tiny


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_of_fp32_to_a_few_roundings(act, rows):
    most = {"gelu": 12.0, "gelu_tanh": 8.0, "silu": 40.0}[act]
    z = torch.linspace(-most, most, 100_003, device="cuda")
    y = rar.linear_forward(torch.ones(rows, 1, device="cuda"), z.view(-1, 1), act=act)
    want, lim = act_and_bound(z.double(), act)
    bad = ~((y.double() - want).abs() <= lim)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, first at z = {float(z[bad.nonzero()[0, 1]])}"


def test_slope_of_fp32_gelu_to_a_few_roundings():
    """cdf + z bell: the function as above, the bell's exponent u, its
    exponential 4u, two products and the fma."""
    z = torch.linspace(-12, 12, 100_003, device="cuda").view(1, -1)
    s = rar.act_backward(torch.ones_like(z), z, "gelu")
    z = z.double()
    q, bell = torch.special.erfc(z.abs() * math.sqrt(0.5)) / 2, torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    want = torch.special.erfc(-z * math.sqrt(0.5)) / 2 + z * bell
    lim = U * (q * (1.3 * z * z + 9.3) + 0.5 * (z > 0) + z.abs() * bell * (z * z / 2 + 7) + want.abs()) + 2.0 ** -145
    bad = ~((s.double() - want).abs() <= lim)
    assert not bool(bad.any()), f"{int(bad.sum())} outside, first at z = {float(z[0, bad.nonzero()[0, 1]])}"


# dtype, whether rows are whole aligned chunks, tile, the output's rows and
# columns (with ragged edges), and sums whose steps of 128 bytes are: three
# whole; four; eight; three, four and eight and a part of one; and one cut into
# parts of several steps
TILED = [("bf16", True, 256, (2312, 3336), (192, 256, 512, 200, 264, 520), (392, 2696, 5128)),
         ("bf16", True, 128, (520, 3592), (192, 256, 512, 200, 264, 520), (136, 1800, 2056)),
         ("bf16", False, 128, (713, 4105), (192, 256, 512, 201, 265, 521), (521, 1161, 2057)),
         ("fp32", True, 128, (712, 4104), (96, 128, 256, 104, 136, 264), (392, 2312, 1032)),
         ("fp32", False, 128, (713, 4105), (96, 128, 256, 105, 137, 265), (521, 1161, 1033))]
TILED = [(dtype, direct, tile, (*out, terms), False) for dtype, direct, tile, out, sums, _ in TILED for terms in sums] + \
        [(dtype, direct, tile, cut, True) for dtype, direct, tile, _, _, cut in TILED]


@pytest.mark.parametrize("dtype, direct, tile, size, in_parts", TILED, ids=str)
@pytest.mark.parametrize("what", ["forward", "input", "weight"])
def test_every_tile_over_many_steps(what, dtype, direct, tile, size, in_parts):
    """The main loop of every tile and loader runs its pairs of whole steps;
    the sizes' cut is asked for, so that other cuts cannot take the cases away."""
    i, j, terms = size
    m, n, k = {"forward": (i, j, terms), "input": (i, terms, j), "weight": (terms, i, j)}[what]
    direction = {"forward": rar.LINEAR_FORWARD, "input": rar.LINEAR_BACKWARD_INPUT, "weight": rar.LINEAR_BACKWARD_WEIGHT}[what]
    got, parts = rar.linear_tiling(direction, m, n, k, dtype, direct)
    assert got == tile and (parts > 1) == in_parts
    step = 64 if dtype == "bf16" else 32
    assert -(-(-(-terms // step)) // parts) >= 3
    layout = (8, 0) if direct else (3, 1)
    if what == "forward":
        forward_case(m, n, k, dtype, "silu", True, True, True, *layout)
    elif what == "input":
        input_case(m, n, k, dtype, "gelu", True, *layout)
    else:
        weight_case(m, n, k, dtype, "fp32", True, True, *layout)
        weight_case(m, n, k, dtype, dtype, False, False, *layout)


def test_a_workspace_of_less_memory_than_elements_is_refused():
    a, b = torch.ones(64, 8192, device="cuda"), torch.ones(64, 8192, device="cuda")
    need = rar.linear_workspace(rar.LINEAR_FORWARD, 64, 64, 8192, "fp32")
    whole = torch.zeros(2 * need, dtype=torch.uint8, device="cuda")
    for bad in (whole[:1].expand(need), whole[::2], torch.empty(need, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace must be"):
            rar.linear_forward(a, b, workspace=bad)
        with pytest.raises(ValueError, match="workspace must be"):
            rar.linear_backward_input(a[:, :64].contiguous(), b, workspace=bad)
        with pytest.raises(ValueError, match="workspace must be"):
            rar.linear_backward_weight(a, b, torch.ones(8192, 8192, device="cuda"), workspace=bad)
    assert not bool(whole.any())
    assert bool((rar.linear_forward(a, b, workspace=whole[:need]) == 8192).all())


@pytest.mark.parametrize("grads", ["fp32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_bias_gradient_of_a_layer_without_inputs(accumulate, grads):
    """bf16 rows of dz summed without a product; whole numbers, so exact."""
    dz = torch.randint(-3, 4, (37, 130), device="cuda").to(torch.bfloat16)
    db = torch.full((130,), 2.0, device="cuda").to(DT[grads])
    rar.linear_backward_weight(dz, dz[:, :0], torch.empty(130, 0, dtype=DT[grads], device="cuda"), db, accumulate=accumulate)
    assert torch.equal(db.float(), dz.float().sum(0) + (2.0 if accumulate else 0.0))
