"""The experts' layers and the losses as a training program uses them
(examples/train_experts.py): it runs, and a micro-batch's gradients are those of
64-bit differentiation of the same weights.

Tolerance: on its way a gradient passes at most 14 roundings to bf16 (h, z0, a, z1, o, y, dz
of two losses, their dy and its sum, dz1, dxs, dh, dz0), each off by 2^-8 at most; the
activations' slopes change by at most twice the relative change of their
arguments. So the difference's norm is below 2 * 14 * 2^-8 of the gradient's."""

import math
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_runs_and_the_ranks_agree():
    import train_experts
    losses = train_experts.main(["--steps", "4", "--vocab", "300", "--tokens", "200", "--experts", "5"])
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)


@pytest.mark.parametrize("tokens", [1, 333])
def test_gradients(tokens):
    import train_experts
    t = train_experts.Trainer(ranks=1, vocab=300, width=72, hidden=104, experts=7)
    batch = train_experts.Corpus(300, seed=4).batch(tokens, padding=0.2 if tokens > 1 else 0.0)
    rank = t.ranks[0]
    for b in (1, 3, 5):   # biases that matter
        rank.low[b].normal_(std=0.3)
    seen = []
    loss = t.gradients(rank, batch, 0.5, False, seen.append)
    t.gradients(rank, batch, 0.5, True, seen.append)   # twice half of it
    assert sorted(seen) == sorted(2 * list(range(7)))
    w = [p.double().requires_grad_(True) for p in rank.low]
    tok, targets, ids, logits = batch
    h = torch.nn.functional.gelu(t.features[tok].double() @ w[0].t() + w[1], approximate="tanh")
    e = t.expert_of[tok]
    a = torch.nn.functional.silu((w[2][e] @ h[:, :, None])[:, :, 0] + w[3][e])
    z = (h + (w[4][e] @ a[:, :, None])[:, :, 0] + w[5][e]) @ w[6].t()
    counts = targets >= 0
    hard = torch.nn.functional.cross_entropy(z[counts], targets[counts])
    q = torch.softmax(logits[counts].double() / t.temperature, 1)
    log_p = torch.log_softmax(z[counts] / t.temperature, 1).gather(1, ids[counts])
    want = hard + t.distill * t.temperature ** 2 * (q * (q.log() - log_p)).sum(1).mean()
    assert abs(float(loss) - float(want.detach())) <= 28 * 2.0 ** -8 * float(want.detach())
    want.backward()
    for p, (g, v) in enumerate(zip(rank.grads, w)):
        off = float((g.double() - v.grad).norm())
        assert off <= 28 * 2.0 ** -8 * float(v.grad.norm()), (p, off, float(v.grad.norm()))
