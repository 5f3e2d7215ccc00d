"""examples/feed_forward.py: the 16-bit linear layer's operators together, as a user
runs them, and the block's gradients against the definition in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import linear as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


def f64(t):
    return t.detach().double().cpu().numpy()


def test_runs():
    block, x = ex.train(steps=5)
    assert all(torch.isfinite(w).all() for w in block.master)
    # a captured step and the eager one before it each moved the offsets
    assert [int(r[1]) for r in block.rng] == [6, 6, 6]
    # the two differ by the order of fp32 sums, which may round h and y, bf16 both, to the
    # other neighbour: one step, 2^-7, of y, and what one step of each h adds through W2
    y, h = block.forward(x, 0.0)
    through = (h[:8].float().abs() @ block.w2.float().abs().t()).max() / y.float().abs().max()
    assert ex.serve(block, x) <= 2.0 ** -7 * (1 + float(through))


def test_gradients():
    """Norms within 2^-6: seven roundings to bf16 in a row (the dropped x, z, h, y, dy, dh and
    dz of each layer), each at most 2^-8 of a value and 2^-9 in the mean square, and the
    result's own."""
    tokens, width, hidden = 96, 136, 264
    block = ex.Block(width, hidden, tokens, p=0.2, seed=3)
    g = torch.Generator("cuda").manual_seed(1)
    x, target = (torch.randn(tokens, width, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    for b in (block.master[1], block.master[3]):
        b.copy_(torch.randn(b.shape, device="cuda", generator=g))
    y, grads = block.gradients(x, target)
    seeds = [tuple(int(v) for v in r) for r in block.rng]
    s = ref.scale(0.2)
    k = [s * ref.keep(tokens, n, 0.2, r) for n, r in zip((width, hidden, width), seeds)]
    X, T, W1, B1, W2, B2 = (f64(t) for t in (x, target, block.w1, block.master[1], block.w2, block.master[3]))
    X = k[0] * X
    Z = X @ W1.T + B1
    H = k[1] * ref.act(Z, "gelu")
    Y = X + k[2] * (H @ W2.T + B2)
    D2 = k[2] * (Y - T) * (2.0 / width)
    D1 = k[1] * (D2 @ W2) * ref.slope(Z, "gelu")
    for what, got, want in zip(("y", "dw1", "db1", "dw2", "db2"), (y, *grads), (Y, D1.T @ X, D1.sum(0), D2.T @ H, D2.sum(0))):
        assert np.linalg.norm(f64(got) - want) <= 2.0 ** -6 * np.linalg.norm(want), what
