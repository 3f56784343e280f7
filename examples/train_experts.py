"""Data-parallel training of a small next-token model with experts over virtual ranks of one GPU.

As in train_mlp.py every rank has its own micro-batches, weights and gradient arena, and the reducer
syncs each bucket as soon as its last gradient is ready. The model is

  h = gelu(f[token] w_in^T + b_in)                    f: fixed features of the tokens
  y = h + w2_e silu(w1_e h + b1_e) + b2_e             e: the token's expert, fixed (hash routing)
  loss = cross entropy of y w_out^T with the next token
         + `distill` times the divergence from a teacher's top logits

The tokens of a micro-batch are sorted by expert on the device, so the experts' layers run as one
launch each and nothing waits for the host. The output layer's logits are never kept.

usage: python examples/train_experts.py [--ranks N] [--steps K] [--vocab V] [--width D] [--experts E] [--tokens M]
"""

import argparse
import os
import sys

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__))]

import torch  # noqa: E402

from train_mlp import Rank  # noqa: E402  (also puts the repository's root on the path)
import ring_all_reduce_ddp_amd as rar  # noqa: E402

ACT, EXPERT_ACT = "gelu_tanh", "silu"


class Corpus:
    """Sequences of a random Markov chain: after token t one of `branch` tokens, the
    k-th with probability in proportion to exp(-k / 2). The teacher knows the chain."""

    def __init__(self, vocab=1000, branch=8, seed=0):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.vocab = vocab
        self.next = torch.stack([torch.randperm(vocab, generator=self.g, device="cuda") for _ in range(branch)], 1)
        self.logits = (-0.5 * torch.arange(branch, device="cuda")).expand(vocab, branch).contiguous()

    def batch(self, tokens, padding=0.1):
        """(tokens, targets, the teacher's ids and logits); some positions are padding, which is not learnt."""
        t = torch.randint(0, self.vocab, (tokens,), generator=self.g, device="cuda")
        k = torch.multinomial(torch.softmax(self.logits[0], 0), tokens, replacement=True, generator=self.g)
        pad = torch.rand(tokens, generator=self.g, device="cuda") < padding
        y = torch.where(pad, -100, self.next[t, k])
        ids = torch.where(pad[:, None], -1, self.next[t])
        return t, y, ids, self.logits[t]


class Trainer:
    def __init__(self, ranks=2, vocab=1000, width=128, hidden=256, experts=8, features=64, seed=0, lr=2e-3, max_norm=1.0,
                 distill=0.5, temperature=2.0):
        self.lr, self.max_norm, self.distill, self.temperature, self.experts = lr, max_norm, distill, temperature, experts
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.features = torch.randn(vocab, features, generator=g, device="cuda").to(torch.bfloat16)
        self.expert_of = torch.randint(0, experts, (vocab,), generator=g, device="cuda")
        shapes = [(width, features), (width,), (experts, hidden, width), (experts, hidden), (experts, width, hidden), (experts, width),
                  (vocab, width)]
        self.shapes = [torch.Size(s) for s in shapes]
        bias = (1, 3, 5)
        initial = [torch.zeros(s, device="cuda") if i in bias else torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5
                   for i, s in enumerate(self.shapes)]
        self.plan = rar.ddp_bucket_plan([s.numel() for s in self.shapes], "fp32", world_size=ranks)
        arena_numel, offsets = self.plan.grad_arena()
        self.ranks = [Rank(self.shapes, offsets, arena_numel, initial) for _ in range(ranks)]
        self.comm = torch.cuda.Stream()
        self.reducer = rar.Reducer(self.plan, [r.grad_arena for r in self.ranks], scale=1.0 / ranks, comm_stream=self.comm)

    def gradients(self, rank, batch, weight, accumulate, ready):
        """Adds the gradients of one micro-batch to the rank's arena and returns its mean loss (on the device);
        ready(p) follows parameter p's. weight: of the micro-batch."""
        w_in, b_in, w1, b1, w2, b2, w_out = rank.low
        g_in, gb_in, g1, gb1, g2, gb2, g_out = rank.grads
        tokens, targets, ids, logits = batch
        # forward
        x = self.features[tokens]
        h, z0 = rar.linear_forward(x, w_in, bias=b_in, act=ACT, keep=True)
        expert = self.expert_of[tokens]
        order = torch.argsort(expert, stable=True)
        back = torch.argsort(order)
        bounds = torch.searchsorted(expert[order], torch.arange(self.experts + 1, device="cuda"))
        xs = h[order]
        a, z1 = rar.experts_forward(xs, w1, bounds, bias=b1, act=EXPERT_ACT, keep=True)
        y = h + rar.experts_forward(a, w2, bounds, bias=b2)[back]
        counts = targets >= 0
        mean = weight * counts / counts.sum().clamp(min=1)
        loss, lse = rar.cross_entropy_forward(y, w_out, targets)
        soft, soft_lse = rar.distill_forward(y, w_out, ids, logits, temperature=self.temperature)
        # backward
        dy = rar.cross_entropy_backward(y, w_out, targets, lse, mean, dw=g_out, accumulate=accumulate)
        dy += rar.distill_backward(y, w_out, ids, logits, soft_lse, self.distill * mean, temperature=self.temperature, dw=g_out,
                                   accumulate=True)
        ready(6)
        do = dy[order]
        rar.experts_backward_weight(do, a, bounds, g2, gb2, accumulate=accumulate)
        ready(5)
        ready(4)
        dz = rar.experts_backward_input(do, w2, bounds, act=EXPERT_ACT, z=z1)
        rar.experts_backward_weight(dz, xs, bounds, g1, gb1, accumulate=accumulate)
        ready(3)
        ready(2)
        dh = dy + rar.experts_backward_input(dz, w1, bounds)[back]
        rar.linear_backward_weight(rar.act_backward(dh, z0, ACT), x, g_in, gb_in, accumulate=accumulate)
        ready(1)
        ready(0)
        return ((loss + self.distill * soft) * mean).sum() / weight

    def step(self, batches):
        """One step; batches[r] is rank r's list of micro-batches. Returns the mean loss."""
        losses = []
        counts = [0] * len(self.shapes)
        self.reducer.prepare()

        def ready(p):
            counts[p] += 1
            if counts[p] == len(self.ranks):   # produced on every rank: its bucket may go
                self.reducer.mark_ready(p)

        for rank, micro in zip(self.ranks, batches):
            for k, batch in enumerate(micro):
                last = k + 1 == len(micro)
                losses.append(self.gradients(rank, batch, 1.0 / len(micro), k > 0, ready if last else (lambda p: None)))
        self.reducer.finalize()
        for rank in self.ranks:
            rank.set.norm(out=rank.norm)
            rank.adamw.step(self.lr, betas=(0.9, 0.95), weight_decay=0.01, max_norm=self.max_norm, norm=rank.norm)
        return torch.stack(losses).mean()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("ranks", 2), ("steps", 60), ("vocab", 1000), ("width", 128), ("hidden", 256), ("experts", 8), ("tokens", 1024),
                          ("micro", 2)):
        ap.add_argument("--" + name, type=int, default=default)
    args = ap.parse_args(argv)
    trainer = Trainer(args.ranks, args.vocab, args.width, args.hidden, args.experts)
    corpus = Corpus(args.vocab)
    losses = []
    for k in range(args.steps):
        loss = trainer.step([[corpus.batch(args.tokens) for _ in range(args.micro)] for _ in trainer.ranks])
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
