"""The AdamW step (include/ddp_train.h) against its formula in 64 bits.

Tolerances, with u = 2^-24 and M = b1 |m| + (1 - b1) |g|, V = b2 v + (1 - b2) g^2
and S = lr / (1 - b1^t) * M / (sqrt(V / (1 - b2^t)) + eps), all in 64 bits:
- the clipped gradient carries 5u (norm, sum, quotient, product, constant);
- m: that, a rounded constant, two products and a sum: 10u M;
- v: twice the gradient's, and as many more: 16u V;
- p: the decay's constant, product and sum, 3u |p|, and of the update the
  moment's 10u M, half of v's 16u, and of the constants, square root (2 with
  margin), sum, quotient (3) and product at most 10u more: 30u S;
- the bf16 weights: the new p rounded once, exactly.
"""

import math

import pytest
import torch

import ring_all_reduce_ddp_amd as rar

from test_gpu_grads import SIZES, U, DT, tensors_of, norm64

pytestmark = pytest.mark.gpu

OPT = {"lr": 2e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1}


def make(numels, dtype, start, steps=0, copy=False, decay=None, seed=20):
    _, g = tensors_of(numels, dtype, seed, start)
    _, p = tensors_of(numels, "fp32", seed + 1, (start + 1) % 4, std=0.02)
    _, m = tensors_of(numels, "fp32", seed + 2, (start + 2) % 4, std=1e-4 if steps else 0.0)
    _, v = tensors_of(numels, "fp32", seed + 3, start, std=1e-4 if steps else 0.0)
    for t in v:
        t.square_()
    c = tensors_of(numels, "bf16", seed + 4, start)[1] if copy else None
    t = torch.full((), steps, dtype=torch.int64, device="cuda")
    s = rar.GradSet(g)
    return s, rar.AdamW(s, p, m, v, t, params_bf16=c, decay=decay)


def step64(opt, o, f, t, decay):
    """The new (p, m, v) and the bounds of their errors, in 64 bits."""
    b1, b2 = o["betas"]
    out = []
    for i, g in enumerate(opt.grads.tensors):
        g = g.double() * f
        p, m, v = (x[i].double() for x in (opt.params, opt.exp_avg, opt.exp_avg_sq))
        mag = b1 * m.abs() + (1 - b1) * g.abs()
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        denom = (v / (1 - b2 ** t)).sqrt() + o["eps"]
        rate = o["lr"] / (1 - b1 ** t)
        wd = o["weight_decay"] if decay is None or decay[i] else 0.0
        new = p - o["lr"] * wd * p - rate * m / denom
        out.append((new, m, v, 3 * U * p.abs() + 30 * U * rate * mag / denom, 10 * U * mag, 16 * U * v))
    return out


def check(opt, want):
    for i, (p, m, v, dp, dm, dv) in enumerate(want):
        assert bool(((opt.params[i].double() - p).abs() <= dp + 2.0 ** -149).all()), f"params[{i}]"
        assert bool(((opt.exp_avg[i].double() - m).abs() <= dm + 2.0 ** -148).all()), f"exp_avg[{i}]"
        assert bool(((opt.exp_avg_sq[i].double() - v).abs() <= dv + 2.0 ** -147).all()), f"exp_avg_sq[{i}]"
        if opt.params_bf16 is not None:
            assert torch.equal(opt.params_bf16[i], opt.params[i].to(torch.bfloat16)), f"params_bf16[{i}]"


@pytest.mark.parametrize("start", [0, 1])
@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", [c for c in SIZES if c != "more tiles than blocks"] + ["large"])
def test_step(case, dtype, copy, start):
    numels = SIZES.get(case, [5_000_003, 4_000_000, 1])
    decay = [i % 3 != 1 for i in range(len(numels))]
    s, opt = make(numels, dtype, start, steps=41, copy=copy, decay=decay)
    norm = s.norm()
    f = min(1.0, 0.01 / (norm64(s.tensors) + 1e-6))
    want = step64(opt, OPT, f, 42, decay)
    opt.step(max_norm=0.01, norm=norm, **OPT)
    check(opt, want)
    assert int(opt.steps) == 42


@pytest.mark.parametrize("steps", [0, 1, 10, 100_000, 2 ** 40])
def test_bias_corrections_and_several_steps(steps):
    s, opt = make([4099, 3], "fp32", 0, steps=steps)
    for k in range(3):
        want = step64(opt, OPT, 1.0, steps + k + 1, None)
        opt.step(**OPT)
        check(opt, want)
        assert int(opt.steps) == steps + k + 1


@pytest.mark.parametrize("change", [{"lr": 0.0}, {"betas": (0.0, 0.0)}, {"betas": (0.95, 0.0)}, {"weight_decay": 0.0},
                                    {"eps": 1e-3}, {"weight_decay": 600.0}])
def test_hyperparameters(change):
    o = {**OPT, **change}
    s, opt = make([10_007], "fp32", 1, steps=3)
    want = step64(opt, o, 1.0, 4, None)
    opt.step(**o)
    check(opt, want)


def test_zero_gradients_and_moments_leave_only_the_decay():
    s, opt = make([1000], "fp32", 0, steps=0)
    s.tensors[0].zero_()
    before = opt.params[0].double()
    opt.step(**OPT)
    assert bool(((opt.params[0].double() - before * (1 - 2e-4)).abs() <= 2 * U * before.abs()).all())


@pytest.mark.parametrize("bad", [math.inf, math.nan, -math.inf])
def test_a_norm_that_is_not_finite_skips_the_step(bad):
    s, opt = make([9001, 5], "fp32", 1, steps=7, copy=True)
    kept = [t.clone() for t in opt.params + opt.exp_avg + opt.exp_avg_sq + opt.params_bf16]
    s.tensors[0][77] = bad
    opt.step(max_norm=1.0, norm=s.norm(), **OPT)
    assert int(opt.steps) == 7
    for a, b in zip(opt.params + opt.exp_avg + opt.exp_avg_sq + opt.params_bf16, kept):
        assert torch.equal(a, b)
    s.tensors[0][77] = 0.0
    want = step64(opt, OPT, min(1.0, 1.0 / (norm64(s.tensors) + 1e-6)), 8, None)
    opt.step(max_norm=1.0, norm=s.norm(), **OPT)
    check(opt, want)
    assert int(opt.steps) == 8


def test_nothing_around_the_tensors_is_written():
    arenas = [torch.full((5003,), math.nan, device="cuda") for _ in range(4)]
    views = [[a[1:4], a[5:4999]] for a in arenas]
    for vs in views:
        for t in vs:
            t.fill_(0.25)
    opt = rar.AdamW(rar.GradSet(views[0]), *views[1:], torch.zeros((), dtype=torch.int64, device="cuda"))
    opt.step(**OPT)
    for a in arenas:
        assert int(torch.isnan(a).sum()) == 5003 - 3 - 4994
    assert torch.equal(arenas[0][5:4999], torch.full((4994,), 0.25, device="cuda"))


def test_graph_of_norm_and_step():
    """Replays move the step count on by themselves and equal eager steps."""
    sizes = [70_001, 33, 8192]
    s, opt = make(sizes, "bf16", 1, steps=0, copy=True, seed=30)
    s2, opt2 = make(sizes, "bf16", 1, steps=0, copy=True, seed=30)
    out = torch.empty((), device="cuda")

    def step(s, opt):
        s.norm(out=out)
        opt.step(max_norm=0.05, norm=out, **OPT)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
            step(s, opt)
    torch.cuda.synchronize()
    for k in range(4):
        step(s2, opt2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert int(opt.steps) == int(opt2.steps) == k + 1
        for a, b in zip(opt.params + opt.exp_avg + opt.exp_avg_sq + opt.params_bf16,
                        opt2.params + opt2.exp_avg + opt2.exp_avg_sq + opt2.params_bf16):
            assert torch.equal(a, b), f"replay {k}"


def test_refusals():
    g, p, m, v = (torch.ones(100, device="cuda") for _ in range(4))
    t = torch.zeros((), dtype=torch.int64, device="cuda")
    s = rar.GradSet([g])
    for args in ([p, p, v], [p, m, m], [g, m, v]):
        with pytest.raises(rar.DDPError, match="overlap"):
            rar.AdamW(s, *[[x] for x in args], t)
    with pytest.raises(ValueError, match="elements"):
        rar.AdamW(s, [p[:99]], [m], [v], t)
    with pytest.raises(ValueError, match="tensors for"):
        rar.AdamW(s, [p, p], [m], [v], t)
    with pytest.raises(ValueError, match="float32"):
        rar.AdamW(s, [p.bfloat16()], [m], [v], t)
    with pytest.raises(ValueError, match="int64"):
        rar.AdamW(s, [p], [m], [v], t.int())
    opt = rar.AdamW(s, [p], [m], [v], t)
    for bad in ({"lr": -1.0}, {"lr": math.nan}, {"eps": -1e-8}, {"weight_decay": -0.1}, {"weight_decay": math.inf}):
        with pytest.raises(rar.DDPError, match="lr, eps"):
            opt.step(**{**OPT, **bad})
    for betas in ((1.0, 0.9), (0.9, 1.0), (-0.1, 0.9), (0.9, math.nan)):
        with pytest.raises(rar.DDPError, match="beta"):
            opt.step(**{**OPT, "betas": betas})
    with pytest.raises(rar.DDPError, match="max_norm"):
        opt.step(max_norm=-1.0, norm=s.norm(), **OPT)
    with pytest.raises(ValueError, match="together"):
        opt.step(max_norm=1.0, **OPT)
    assert int(t) == 0 and bool((p == 1).all())


def test_a_norm_inside_the_state_is_refused():
    g, p, m, v = (torch.ones(100, device="cuda") for _ in range(4))
    c = torch.ones(100, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros((), dtype=torch.int64, device="cuda")
    opt = rar.AdamW(rar.GradSet([g]), [p], [m], [v], t, params_bf16=[c])
    for inside, what in ((p[0], "params"), (m[99], "exp_avg"), (v[50], "exp_avg_sq"), (c.view(torch.float32)[49], "params_bf16"),
                         (t.view(1).view(torch.float32)[1], "step_dev")):
        with pytest.raises(rar.DDPError, match="norm_dev and " + what):
            opt.step(max_norm=1.0, norm=inside, **OPT)
    assert int(t) == 0 and bool((p == 1).all())
    opt.step(max_norm=1.0, norm=g[3], **OPT)   # the gradients are only read
    assert int(t) == 1


@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_step_beyond_the_cache(dtype, copy):
    """More than the Infinity Cache (256 MiB) of gradients and state: every access is streamed."""
    numels = [20_000_003, 511, 3, 5_000_001]
    decay = [True, False, True, False]
    s, opt = make(numels, dtype, 1, steps=41, copy=copy, decay=decay)
    want = step64(opt, OPT, min(1.0, 0.01 / (norm64(s.tensors) + 1e-6)), 42, decay)
    opt.step(max_norm=0.01, norm=s.norm(), **OPT)
    check(opt, want)
    assert int(opt.steps) == 42
