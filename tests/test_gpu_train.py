"""The training step that runs the operators together (examples/train_mlp.py):
its gradients against 64-bit differentiation of the same model, the ranks'
agreement, and the loss."""

import math
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

import train_mlp  # noqa: E402

pytestmark = pytest.mark.gpu


def model64(weights, blocks, x):
    gelu = lambda z: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))  # noqa: E731
    h = gelu(x @ weights[0].t() + weights[1])
    for k in range(blocks):
        w1, b1, w2, b2 = weights[2 + 4 * k:6 + 4 * k]
        h = h + gelu(h @ w1.t() + b1) @ w2.t() + b2
    return h @ weights[-2].t() + weights[-1]


def test_gradients_of_a_step():
    """Two ranks, two micro-batches each: every parameter's synced gradient is the
    mean over all rows of the 64-bit gradient at the bf16 weights. Activations and
    the gradients between layers are rounded to bf16 (relative error 2^-8 at most, about 2^-9.5 in the
    mean square) some 4 times on each way through 2 blocks, forward and back, and independently from element to
    element: below 12 * 2^-9.5 of the gradient's norm with room to spare; 3 % is asked."""
    t = train_mlp.Trainer(ranks=2, width=64, hidden=136, blocks=2, features=24, outputs=9, lr=0.0)
    batch = train_mlp.teacher(24, 9, seed=3)
    batches = [[batch(77), batch(77)] for _ in range(2)]
    for r in t.ranks:   # biases away from zero, the same on each rank
        for i, b in enumerate(r.low):
            if b.dim() == 1:
                b.copy_(torch.sin(torch.arange(b.numel(), device="cuda") + i) * 0.2)
    weights = [w.double().requires_grad_(True) for w in t.ranks[0].low]
    t.step(batches)
    loss = 0.0
    for micro in batches:
        for x, target in micro:
            loss = loss + (model64(weights, 2, x.double()) - target.double()).square().mean() / 4
    want = torch.autograd.grad(loss, weights)
    total = 0.0
    for i, (g, w) in enumerate(zip(t.ranks[0].grads, want)):
        total += float(w.square().sum())
        assert float((g.double() - w).norm()) <= 0.03 * float(w.norm()), f"parameter {i}"
        assert torch.equal(g, t.ranks[1].grads[i]), f"parameter {i} differs between the ranks"
    assert abs(float(t.ranks[0].norm) - math.sqrt(total)) <= 0.03 * math.sqrt(total)


def test_training_lowers_the_loss_and_keeps_the_ranks_equal():
    losses = train_mlp.main(["--ranks", "3", "--steps", "40", "--width", "128", "--hidden", "256", "--blocks", "1", "--rows", "200"])
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < 0.5 * losses[0]
