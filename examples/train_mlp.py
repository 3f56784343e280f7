"""Data-parallel training of a small residual MLP over virtual ranks of one GPU.

Every rank has its own micro-batches, weights and gradient arena. A step is

  forward     bf16 linear layers; bias, activation and residual in the product's pass
  backward    input gradients through the activations; weight and bias gradients summed over
              the micro-batches in fp32, straight into the rank's gradient arena
  sync        the reducer reduces each bucket in place as soon as its last gradient is ready
  update      the global gradient norm, and AdamW on fp32 master weights with the clipping
              factor read on the device; it writes the bf16 weights of the next forward pass

usage: python examples/train_mlp.py [--ranks N] [--steps K] [--width D] [--hidden H] [--blocks L] [--rows M]
"""

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import ring_all_reduce_ddp_amd as rar  # noqa: E402

ACT = "gelu_tanh"


class Rank:
    """One rank's arenas (gradients, fp32 weights, moments, bf16 weights) and its optimizer."""

    def __init__(self, shapes, offsets, arena_numel, initial):
        arena = lambda dtype=torch.float32: torch.zeros(arena_numel, dtype=dtype, device="cuda")  # noqa: E731
        views = lambda a: [a[o:o + s.numel()].view(s) for o, s in zip(offsets, shapes)]  # noqa: E731
        self.grad_arena = arena()
        self.grads, self.weights, self.m, self.v = views(self.grad_arena), views(arena()), views(arena()), views(arena())
        self.low = views(arena(torch.bfloat16))
        for w, c, x in zip(self.weights, self.low, initial):
            w.copy_(x)
            c.copy_(x)
        self.steps = torch.zeros((), dtype=torch.int64, device="cuda")
        self.norm = torch.zeros((), device="cuda")
        self.set = rar.GradSet(self.grads)
        self.adamw = rar.AdamW(self.set, self.weights, self.m, self.v, self.steps, params_bf16=self.low,
                               decay=[len(s) > 1 for s in shapes])


class Trainer:
    """An input layer x -> gelu(x w^T + b), `blocks` of h + w2 gelu(w1 h + b1) + b2, and an output layer."""

    def __init__(self, ranks=4, width=256, hidden=1024, blocks=2, features=64, outputs=32, seed=0, lr=1e-3, max_norm=1.0):
        self.blocks, self.lr, self.max_norm = blocks, lr, max_norm
        shapes = [(width, features), (width,)]
        for _ in range(blocks):
            shapes += [(hidden, width), (hidden,), (width, hidden), (width,)]
        shapes += [(outputs, width), (outputs,)]
        self.shapes = [torch.Size(s) for s in shapes]
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        initial = [torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5 if len(s) > 1 else torch.zeros(s, device="cuda")
                   for s in self.shapes]
        self.plan = rar.ddp_bucket_plan([s.numel() for s in self.shapes], "fp32", world_size=ranks)
        arena_numel, offsets = self.plan.grad_arena()
        self.ranks = [Rank(self.shapes, offsets, arena_numel, initial) for _ in range(ranks)]
        self.comm = torch.cuda.Stream()
        self.reducer = rar.Reducer(self.plan, [r.grad_arena for r in self.ranks], scale=1.0 / ranks, comm_stream=self.comm)

    def forward(self, rank, x):
        """The output, and what the backward pass needs."""
        w = rank.low
        h, z0 = rar.linear_forward(x, w[0], bias=w[1], act=ACT, keep=True)
        kept = [(x, z0)]
        for k in range(self.blocks):
            w1, b1, w2, b2 = w[2 + 4 * k:6 + 4 * k]
            a, z = rar.linear_forward(h, w1, bias=b1, act=ACT, keep=True)
            kept.append((h, a, z))
            h = rar.linear_forward(a, w2, bias=b2, residual=h)
        kept.append(h)
        return rar.linear_forward(h, w[-2], bias=w[-1]), kept

    def backward(self, rank, dy, kept, accumulate, ready):
        """Adds the gradients of one micro-batch to the rank's arena; ready(p) follows parameter p's."""
        w, g = rank.low, rank.grads
        n = len(w)

        def weight(i, dz, x):
            rar.linear_backward_weight(dz, x, g[i], g[i + 1], accumulate=accumulate)
            ready(i + 1)
            ready(i)

        weight(n - 2, dy, kept[-1])
        dh = rar.linear_backward_input(dy, w[n - 2])
        for k in reversed(range(self.blocks)):
            h, a, z = kept[1 + k]
            i = 2 + 4 * k
            weight(i + 2, dh, a)
            dz = rar.linear_backward_input(dh, w[i + 2], act=ACT, z=z)
            weight(i, dz, h)
            dh = rar.linear_backward_input(dz, w[i], add=dh)
        x, z0 = kept[0]
        weight(0, rar.act_backward(dh, z0, ACT), x)

    def step(self, batches):
        """One step; batches[r] is rank r's list of micro-batches (x, target). Returns the mean loss."""
        losses = []
        counts = [0] * len(self.shapes)
        self.reducer.prepare()

        def ready(p):
            counts[p] += 1
            if counts[p] == len(self.ranks):   # produced on every rank: its bucket may go
                self.reducer.mark_ready(p)

        for rank, micro in zip(self.ranks, batches):
            for k, (x, target) in enumerate(micro):
                y, kept = self.forward(rank, x)
                diff = y.float() - target
                losses.append(diff.square().mean())
                dy = (diff * (2.0 / diff.numel() / len(micro))).to(torch.bfloat16)
                last = k + 1 == len(micro)
                self.backward(rank, dy, kept, k > 0, ready if last else (lambda p: None))
        self.reducer.finalize()
        for rank in self.ranks:
            rank.set.norm(out=rank.norm)
            rank.adamw.step(self.lr, betas=(0.9, 0.95), weight_decay=0.01, max_norm=self.max_norm, norm=rank.norm)
        return torch.stack(losses).mean()


def teacher(features, outputs, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.randn(outputs, features, generator=g, device="cuda") * features ** -0.5

    def batch(rows):
        x = torch.randn(rows, features, generator=g, device="cuda").to(torch.bfloat16)
        return x, torch.sin(2.0 * (x.float() @ t.t()))
    return batch


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("ranks", 4), ("steps", 60), ("width", 256), ("hidden", 1024), ("blocks", 2), ("rows", 512), ("micro", 2)):
        ap.add_argument("--" + name, type=int, default=default)
    args = ap.parse_args(argv)
    trainer = Trainer(args.ranks, args.width, args.hidden, args.blocks)
    batch = teacher(64, 32, seed=1)
    losses = []
    for k in range(args.steps):
        loss = trainer.step([[batch(args.rows) for _ in range(args.micro)] for _ in trainer.ranks])
        losses.append(float(loss))
        if k % 10 == 0 or k + 1 == args.steps:
            print(f"step {k}: loss {losses[-1]:.4f}, gradient norm {float(trainer.ranks[0].norm):.4f}", flush=True)
    first = trainer.ranks[0]
    for rank in trainer.ranks[1:]:
        for a, b in zip(first.weights, rank.weights):
            if not torch.equal(a, b):
                raise SystemExit("the ranks' weights differ")
    print("the ranks' weights are equal bit for bit")
    return losses


if __name__ == "__main__":
    main()
