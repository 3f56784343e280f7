"""The operators around the sync where one launch cannot hold their blocks: a
dispatch has fewer than 2^32 threads, 2^24 blocks of 256. Up to 120 GB of HBM."""

import pytest
import torch

import ring_all_reduce_ddp_amd as rar

pytestmark = pytest.mark.gpu

BLOCKS = 1 << 24


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def all_equal(t, value):
    """Whether every element of a long vector is `value`, a part at a time."""
    part = 1 << 31
    return all(bool((t[k:k + part] == value).all()) for k in range(0, t.numel(), part))


def test_clip_of_more_parts_than_a_launch_has_blocks():
    """Blocks of 2048 elements; an element scaled twice or not at all shows."""
    n = BLOCKS * 2048 + 2049
    t = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    print(f"[clip] {n} elements", flush=True)
    rar.GradSet([t]).clip(1.0, torch.full((), 4.0, device="cuda"))
    assert all_equal(t, 0.25)   # 1 / 4.000001 rounds to it


def test_adamw_of_more_tiles_than_a_launch_has_blocks():
    """Blocks of 512 elements, fp32 state and bf16 gradients (120 GB). Every
    element's first step is checked: m = (1 - b1) g and v = (1 - b2) g^2 as they
    are rounded, p one lr away."""
    n = BLOCKS * 512 + 513
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    steps = torch.zeros((), dtype=torch.int64, device="cuda")
    opt = rar.AdamW(rar.GradSet([g]), [p], [m], [v], steps)
    print(f"[adamw] {n} elements", flush=True)
    opt.step(0.25, betas=(0.5, 0.75), eps=0.0, weight_decay=0.0)
    assert int(steps) == 1
    # the moments are exact, their corrections 1/2 and 1/4 and p = -lr but for a few roundings
    assert all_equal(m, 0.25) and all_equal(v, 0.0625)
    assert all_equal(p, float(p[0])) and abs(float(p[0]) + 0.25) <= 0.25 * 8 * 2.0 ** -24
    opt.step(0.25, betas=(0.5, 0.75), eps=0.0, weight_decay=0.0)
    assert int(steps) == 2
    assert all_equal(m, 0.375) and all_equal(v, 0.109375)


def whole(shape, most):
    """Whole numbers in [-most, most], small enough that bf16 and the sums below hold them exactly."""
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").random_(0, 2 * most + 1).sub_(most)


def test_few_rows_of_more_outputs_than_a_launch_has_blocks():
    """Blocks of four outputs."""
    n, k = BLOCKS * 4 + 5, 8
    x, w = whole((1, k), 2), whole((n, k), 2)
    print(f"[few rows] {n} outputs", flush=True)
    y = rar.linear_forward(x, w)
    assert torch.equal(y[0], (w * x).sum(1))


def test_products_of_more_tiles_than_a_launch_has_blocks():
    """Tiles of 64 rows and one column: forward, input gradient, weight and bias gradient."""
    m = BLOCKS * 64 + 65
    tall, one, dz = whole((m, 1), 9), whole((1, 1), 9), whole((1, m), 9)
    print(f"[tiles] {m} rows", flush=True)
    assert torch.equal(rar.linear_forward(tall, one), tall * one)
    assert torch.equal(rar.linear_backward_input(tall, one), tall * one)
    dw, db = torch.empty_like(tall), torch.empty(m, dtype=torch.bfloat16, device="cuda")
    rar.linear_backward_weight(dz, one, dw, db)
    assert torch.equal(dw, dz.t() * one) and torch.equal(db, dz[0])
