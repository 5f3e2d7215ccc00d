"""Train a feed-forward block with dropout in one captured graph, and serve it:
every operator of include/hkg_linear.h in the place it is made for.

    python examples/feed_forward.py [--steps 200]

The block y = x + D2(W2 D1(gelu(W1 x + b1)) + b2) learns a random teacher's
outputs from inputs that it sees through dropout.  A step
  1. drops elements of the inputs;
  2. forms y with two products, which apply everything else as they store;
  3. forms the loss's gradient dy in bf16, and from it all others, with the masks
     of step 2 computed again;
  4. moves fp32 master weights, and rounds them to bf16 for the next step;
  5. moves the generator's offset, so that the next replay draws other masks.
All of it is one graph: a step is one launch for the host.  After training the
block answers single tokens, which must agree with the whole batch.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_gemm_fp8_amd as hkg  # noqa: E402


class Block:
    def __init__(self, width, hidden, tokens, p=0.1, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.p = p
        # a call's masks depend on (seed, offset): one seed a place, one offset a step
        self.rng = [torch.tensor([seed + 1 + i, 0], dtype=torch.int64, device="cuda") for i in range(3)]
        self.master = [torch.randn(hidden, width, device="cuda", generator=g) / width ** 0.5, torch.zeros(hidden, device="cuda"),
                       torch.randn(width, hidden, device="cuda", generator=g) / hidden ** 0.5, torch.zeros(width, device="cuda")]
        self.w1, self.w2 = (self.master[i].to(torch.bfloat16) for i in (0, 2))
        self.z = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")

    def forward(self, x, p, z=None):
        """-> (y, the hidden values that the second product read)."""
        r = self.rng if p else [None] * 3
        h = hkg.linear(x, self.w1, self.master[1], activation="gelu", p=p, rng=r[1], z=z)
        return hkg.linear(h, self.w2, self.master[3], residual=x, p=p, rng=r[2]), h

    def gradients(self, x, target):
        """-> y, and the gradients of mean (y - target)^2 times tokens for the master weights."""
        x = hkg.dropout(x, self.p, self.rng[0])
        y, h = self.forward(x, self.p, self.z)
        dy = (y - target) * (2.0 / y.shape[1])
        dh, dw2, db2 = hkg.linear_backward(dy, h, self.w2, p=self.p, rng=self.rng[2])
        _, dw1, db1 = hkg.linear_backward(dh, x, self.w1, z=self.z, activation="gelu", p=self.p, rng=self.rng[1], need_dx=False)
        return y, (dw1, db1, dw2, db2)

    def step(self, x, target, lr):
        _, grads = self.gradients(x, target)
        for w, d in zip(self.master, grads):
            w.sub_(d, alpha=lr / x.shape[0])
        self.w1.copy_(self.master[0])
        self.w2.copy_(self.master[2])
        for r in self.rng:
            r[1:].add_(1)


def train(tokens=512, width=256, hidden=1024, steps=200, lr=2.0, seed=0, log=print):
    """-> (the block, x)."""
    g = torch.Generator("cuda").manual_seed(seed + 100)
    x = torch.randn(tokens, width, device="cuda", generator=g).to(torch.bfloat16)
    teacher = Block(width, hidden, tokens, seed=seed + 50)
    target, _ = teacher.forward(x, 0.0)
    block = Block(width, hidden, tokens, seed=seed)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                              # a first step outside of the graph
        block.step(x, target, lr)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, target, lr)

    def loss():
        return float((block.forward(x, 0.0)[0] - target).float().square().mean())
    first = loss()
    for _ in range(steps):
        graph.replay()
    log("loss without dropout %.4f -> %.4f over %d steps" % (first, loss(), steps))
    return block, x


def serve(block, x, log=print):
    """The first tokens one by one against the whole batch -> largest difference,
    relative to the largest y."""
    y = block.forward(x, 0.0)[0].float()
    got = torch.cat([block.forward(x[i:i + 1], 0.0)[0] for i in range(8)]).float()
    off = float((got - y[:8]).abs().max() / y.abs().max())
    log("tokens one by one: within %.1e of the batch" % off)
    return off


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    serve(*train(steps=a.steps))


if __name__ == "__main__":
    main()
