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
