"""The global gradient norm and clipping (include/ddp_train.h) against plain
64-bit arithmetic.

Tolerances, with u = 2^-24 (fp32) and b = 2^-8 (bf16), the largest relative
errors of one rounding to nearest:
- norm: summed in fp64, so one rounding to fp32: u (and 1e-12 for the sum);
- max norm: exact;
- clipped: the factor max_norm / (norm + 1e-6) has the norm's u, one of the
  sum, one of the quotient (and the constant's, smaller), and the product
  rounds once more: 5u, and b if the result is bf16. Results below the
  smallest normal number also lose up to one subnormal step.
"""

import math

import pytest
import torch

import ring_all_reduce_ddp_amd as rar

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZES = {
    "one element": [1],
    "nothing": [],
    "empty tensors": [0, 5, 0],
    "one tile": [8192],
    "one tile and one": [8193],
    "ragged": [3, 8191, 8192, 16385, 1, 0, 7, 2],
    "many": [1 + (37 * i) % 61 for i in range(700)],
    "more tiles than blocks": [2049 * 8192 + 3, 11],
}


def tensors_of(numels, dtype, seed, start=0, std=1e-3):
    """Views into one arena, tensor after tensor without gaps, the first one
    `start` elements into it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    arena = (torch.randn(start + sum(numels) + 8, generator=g, device="cuda") * std).to(DT[dtype])
    out, at = [], start
    for m in numels:
        out.append(arena[at:at + m])
        at += m
    return arena, out


def norm64(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


@pytest.mark.parametrize("start", [0, 1, 3])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", SIZES)
def test_norm(case, dtype, start):
    _, ts = tensors_of(SIZES[case], dtype, 5, start)
    s = rar.GradSet(ts)
    got = s.norm()
    want = norm64(ts)
    assert abs(float(got) - want) <= (U + 1e-12) * want
    again = s.norm()
    assert torch.equal(got, again), "a repeated call gives the same bits"
    most = max([float(t.abs().max()) for t in ts if t.numel()], default=0.0)
    assert float(s.norm("max")) == most


@pytest.mark.parametrize("value,dtype", [(1e30, "fp32"), (1e-30, "fp32"), (1e-42, "fp32"), (3e38, "bf16")])
def test_norm_of_values_whose_squares_leave_fp32(value, dtype):
    t = torch.full((10_001,), value, device="cuda").to(DT[dtype])
    want = norm64([t])
    if want > torch.finfo(torch.float32).max:
        want = math.inf
    got = float(rar.GradSet([t]).norm())
    # a subnormal result is spaced 2^-149
    assert got == want or abs(got - want) <= U * 1.001 * want + 2.0 ** -149


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("at", [0, 8191, 8192, 20_000])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_of_values_that_are_not_finite(dtype, at, kind):
    _, ts = tensors_of([20_001], dtype, 6)
    s = rar.GradSet(ts)
    ts[0][at] = -math.inf
    assert float(s.norm(kind)) == math.inf
    ts[0][(at + 1) % 20_001] = math.nan
    assert math.isnan(float(s.norm(kind)))
    ts[0][at] = 0.0
    assert math.isnan(float(s.norm(kind)))


def test_norm_beyond_32_bit_offsets():
    """More than 2^32 bytes and 2^31 elements in one tensor, with the values at its far end."""
    n = 2 ** 31 + 8192 + 5
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-3:] = 2.0
    t[2 ** 31] = 1.0
    assert float(rar.GradSet([t]).norm()) == pytest.approx(math.sqrt(13.0), rel=1e-7)
    into = torch.empty_like(t)
    dst = rar.GradSet([into])
    src = rar.GradSet([t])
    src.clip(1.0, src.norm(), into=dst)
    assert into[-3:].float().tolist() == pytest.approx([2 / math.sqrt(13.0)] * 3, rel=B)
    assert int(torch.count_nonzero(into)) == 4


def check_clipped(got, given, norm, max_norm, dtype):
    f = min(1.0, max_norm / (norm + 1e-6)) if not math.isinf(max_norm) else 1.0
    for x, g in zip(got, given):
        want = g.double() * f
        tol = (5 * U + (B if dtype == "bf16" else 0.0)) * want.abs() + (2.0 ** -133 if dtype == "bf16" else 2.0 ** -149)
        assert bool(((x.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("start", [0, 1])
@pytest.mark.parametrize("pair", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("case", SIZES)
def test_clip_into(case, pair, start):
    _, ts = tensors_of(SIZES[case], pair[0], 7, start)
    arena, into = tensors_of(SIZES[case], pair[1], 8, 2 - start)
    outside = [arena[:2 - start].clone(), arena[2 - start + sum(SIZES[case]):].clone()]
    before = [t.clone() for t in ts]
    s, d = rar.GradSet(ts), rar.GradSet(into)
    norm = s.norm()
    s.clip(0.01, norm, into=d)
    check_clipped(into, before, float(norm), 0.01, pair[1])
    for t, b in zip(ts, before):
        assert torch.equal(t, b), "the gradients stay"
    assert torch.equal(arena[:2 - start], outside[0])
    assert torch.equal(arena[2 - start + sum(SIZES[case]):], outside[1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("max_norm", [0.0, 0.01, 1e4, math.inf])
def test_clip_in_place(max_norm, dtype):
    _, ts = tensors_of(SIZES["ragged"], dtype, 9, 1)
    before = [t.clone() for t in ts]
    s = rar.GradSet(ts)
    norm = s.norm()
    s.clip(max_norm, norm)
    if max_norm >= 1e4:
        assert all(torch.equal(t, b) for t, b in zip(ts, before))
    else:
        check_clipped(ts, before, float(norm), max_norm, dtype)


def test_clip_by_a_norm_that_is_not_finite():
    _, ts = tensors_of([9000], "fp32", 10)
    _, into = tensors_of([9000], "fp32", 11)
    s, d = rar.GradSet(ts), rar.GradSet(into)
    s.clip(1.0, torch.tensor(math.inf, device="cuda"), into=d)
    assert bool((into[0] == 0).all())
    s.clip(1.0, torch.tensor(math.nan, device="cuda"), into=d)
    assert bool(torch.isnan(into[0]).all())


def test_arena_padding_is_not_read():
    """The gaps between an arena's members are not gradients: what lies there
    changes neither the norm nor is it written."""
    plan = rar.ddp_bucket_plan([5, 9, 1, 4097], "fp32", world_size=1)
    length, offs = plan.grad_arena()
    arena = torch.full((length,), math.nan, device="cuda")
    ts = [arena[o:o + m] for o, m in zip(offs, [5, 9, 1, 4097])]
    for t in ts:
        t.fill_(0.5)
    s = rar.GradSet(ts)
    norm = s.norm()
    assert float(norm) == pytest.approx(0.5 * math.sqrt(4112), rel=1e-7)
    s.clip(1.0, norm)
    assert int(torch.isnan(arena).sum()) == length - 4112


def test_on_another_stream():
    """The calls run on the stream they are given, in its order."""
    side = torch.cuda.Stream()
    _, ts = tensors_of([3_000_001, 17], "fp32", 12)
    s = rar.GradSet(ts)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in ts:
            t.mul_(2.0)
    norm = s.norm(stream=side)
    s.clip(1.0, norm, stream=side)
    after = s.norm(stream=side)
    side.synchronize()
    assert float(after) == pytest.approx(1.0, rel=1e-5)
    assert float(norm) == pytest.approx(1e-3 * 2 * math.sqrt(3_000_018), rel=1e-2)


def test_graph_of_norm_and_clip():
    _, ts = tensors_of(SIZES["ragged"] + [100_003], "fp32", 13, 1)
    pristine = [t.clone() for t in ts]
    s = rar.GradSet(ts)
    out = torch.empty((), device="cuda")

    def step():
        s.norm(out=out)
        s.clip(0.01, out)

    step()
    torch.cuda.synchronize()
    want, want_norm = [t.clone() for t in ts], out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
            step()
    for _ in range(4):
        for t, p in zip(ts, pristine):
            t.copy_(p)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_norm)
        assert all(torch.equal(t, w) for t, w in zip(ts, want))


def test_refusals():
    t = torch.ones(100, device="cuda")
    with pytest.raises(rar.DDPError, match="overlap"):
        rar.GradSet([t[:60], t[59:]])
    with pytest.raises(ValueError, match="contiguous"):
        rar.GradSet([t[::2]])
    with pytest.raises(ValueError, match="contiguous"):
        rar.GradSet([t, t.bfloat16()])
    with pytest.raises(ValueError):
        rar.GradSet([torch.ones(3)])
    s = rar.GradSet([t])
    norm = s.norm()
    with pytest.raises(rar.DDPError, match="max_norm"):
        s.clip(-1.0, norm)
    with pytest.raises(rar.DDPError, match="max_norm"):
        s.clip(math.nan, norm)
    with pytest.raises(rar.DDPError, match="element counts"):
        s.clip(1.0, norm, into=rar.GradSet([torch.ones(99, device="cuda")]))
    with pytest.raises(rar.DDPError, match="overlap"):
        s.clip(1.0, norm, into=rar.GradSet([t]))
    big = torch.ones(40, device="cuda")
    a, b = rar.GradSet([big[:10], big[20:30]]), rar.GradSet([big[10:20], big[25:35]])
    with pytest.raises(rar.DDPError, match="overlap"):
        a.clip(1.0, norm, into=b)
    a.clip(1.0, norm, into=rar.GradSet([big[10:20], big[30:40]]))   # interleaved, but apart
    with pytest.raises(ValueError, match="float32"):
        s.norm(out=torch.empty((), dtype=torch.float64, device="cuda"))
    with pytest.raises(KeyError):
        s.norm("l1")


def test_a_freed_set_is_refused():
    a, b = (torch.full((10,), 4.0, device="cuda") for _ in range(2))
    s, into = rar.GradSet([a]), rar.GradSet([b])
    norm = s.norm()
    into.free()
    with pytest.raises(ValueError, match="into is freed"):   # not in place
        s.clip(1.0, norm, into=into)
    with pytest.raises(rar.DDPError, match="grads is NULL"):
        into.norm()
    assert (a == 4.0).all() and (b == 4.0).all()


def test_a_norm_inside_what_is_written_is_refused():
    big = torch.ones(100, device="cuda")
    s, into = rar.GradSet([big[10:20], big[40:60]]), rar.GradSet([big[20:30], big[70:90]])
    norm = s.norm(out=big[25])   # another set's tensor is none of the norm's business
    for at in (10, 19, 40, 59):
        with pytest.raises(rar.DDPError, match="norm_dev and grads"):
            s.norm(out=big[at])
        with pytest.raises(rar.DDPError, match="norm_dev and grads"):
            s.clip(1.0, big[at])
    for at in (20, 25, 89):
        with pytest.raises(rar.DDPError, match="norm_dev and grads"):
            s.clip(1.0, big[at], into=into)
    assert float(norm) == pytest.approx(math.sqrt(30.0), rel=U) and int((big == 1).sum()) == 99
    for at in (9, 39, 60, 99):
        s.norm(out=big[at])
    s.clip(1.0, big[45], into=into)   # among the gradients, which are only read
    f = 1 / (1 + 1e-6)
    assert ((into.tensors[0].double() - f).abs() <= 5 * U).all() and ((into.tensors[1].double() - f).abs() <= 5 * U).all()


# more than the Infinity Cache (256 MiB) in either type, with odd starts and ends
BEYOND_THE_CACHE = [70_000_001, 8191, 70_000_003, 5]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_beyond_the_cache(dtype):
    """Both norms' streamed loads."""
    _, ts = tensors_of(BEYOND_THE_CACHE, dtype, 14, 1)
    s = rar.GradSet(ts)
    want = norm64(ts)
    assert abs(float(s.norm()) - want) <= (U + 1e-12) * want
    assert float(s.norm("max")) == max(float(t.abs().max()) for t in ts)


@pytest.mark.parametrize("pair", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp32"), ("bf16", "bf16")])
def test_clip_into_beyond_the_cache(pair):
    _, ts = tensors_of(BEYOND_THE_CACHE, pair[0], 15, 1)
    arena, into = tensors_of(BEYOND_THE_CACHE, pair[1], 16, 2)
    outside = [arena[:2].clone(), arena[2 + sum(BEYOND_THE_CACHE):].clone()]
    s, d = rar.GradSet(ts), rar.GradSet(into)
    norm = s.norm()
    s.clip(0.01, norm, into=d)
    check_clipped(into, ts, float(norm), 0.01, pair[1])
    assert torch.equal(arena[:2], outside[0]) and torch.equal(arena[2 + sum(BEYOND_THE_CACHE):], outside[1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_clip_in_place_beyond_the_cache(dtype):
    _, ts = tensors_of(BEYOND_THE_CACHE, dtype, 17, 1)
    before = [t.clone() for t in ts]
    s = rar.GradSet(ts)
    norm = s.norm()
    s.clip(0.01, norm)
    check_clipped(ts, before, float(norm), 0.01, dtype)
    for t, b in zip(ts, before):
        t.copy_(b)
    s.clip(1e4, norm)
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
