"""Train one linear layer in MXFP4 and serve it: every operator of
include/hkg_ops.h in the place it is made for.

    python examples/mxfp4_linear.py [--steps 60]

A layer y = x W^T learns a random teacher's outputs.  A step
  1. quantises W and x, each along its rows and (for the gradients) along its
     columns, in one pass over each;
  2. forms y with the MXFP4 product and the loss's gradient dy in fp32;
  3. forms the weight's gradient from dy and x^T in MXFP4;
  4. adds it to an fp32 momentum, orthogonalises that and moves W.
After training the layer answers single tokens and a small batch through the
few-token form, which must agree with the product over the whole batch.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_gemm_fp8_amd as hkg  # noqa: E402

A, B = hkg.HKG_MX_OPERAND_A, hkg.HKG_MX_OPERAND_B


def train(tokens=1024, n=512, k=768, steps=60, lr=0.12, momentum=0.9, seed=0, log=print):
    """-> (first loss, last loss, trained W in fp32, x)."""
    g = torch.Generator("cuda").manual_seed(seed)
    teacher = torch.randn(n, k, device="cuda", generator=g) / k ** 0.5
    x = torch.randn(tokens, k, device="cuda", generator=g).to(torch.bfloat16)
    target = x.float() @ teacher.t()
    W = torch.zeros(n, k, device="cuda")                      # fp32 master weights
    buf = torch.zeros_like(W)
    xq, xs, xt, xts = hkg.mxfp4_quantize_both(x, A, B)         # one batch: its forms are kept
    losses = []
    for step in range(steps):
        wq, ws, wt, wts = hkg.mxfp4_quantize_both(W, B, B)
        y = hkg.gemm_mxfp4(xq, wq, xs, ws).float()
        loss = (y - target).square().mean()
        dy = (y - target) * (2.0 / target.numel())
        _, dw = hkg.linear_mxfp4_backward(dy, wt, wts, xt, xts)   # dx would go on to the layer before
        buf.mul_(momentum).add_(dw.float())
        # a unit-spectrum step, scaled to the layer's shape and cooled down linearly;
        # all of them together, lr steps / 2 (n / k)^1/2 = 2.9, have to exceed the
        # teacher's largest singular value, 1 + (n / k)^1/2 = 1.8
        W.add_(hkg.orthogonalize(buf).float(), alpha=-lr * (1.0 - step / steps) * (n / k) ** 0.5)
        losses.append(loss)
    losses = [float(v) for v in losses]
    log("loss %.4f -> %.4f over %d steps" % (losses[0], losses[-1], steps))
    return losses[0], losses[-1], W, x


def serve(W, x, log=print):
    """Answers of the trained layer for single tokens and a batch of 16 against
    the product over all tokens -> largest difference, relative to the largest y."""
    wq, ws = hkg.mxfp4_quantize(W, B)
    xq, xs = hkg.mxfp4_quantize(x, A)
    y = hkg.gemm_mxfp4(xq, wq, xs, ws).float()
    got = torch.cat([hkg.linear_mxfp4(x[i:i + 1], wq, ws) for i in range(8)] + [hkg.linear_mxfp4(x[8:24], wq, ws)] +
                    [hkg.linear_mxfp4(x[24:], wq, ws)]).float()
    off = float((got - y).abs().max() / y.abs().max())
    log("tokens one by one, a batch of 16, the rest: within %.1e of the product over all" % off)
    return off


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    _, _, W, x = train(steps=a.steps)
    serve(W, x)


if __name__ == "__main__":
    main()
