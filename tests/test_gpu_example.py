"""examples/mxfp4_linear.py: the operators together, as a user runs them."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_trains_and_serves():
    spec = importlib.util.spec_from_file_location("mxfp4_linear", os.path.join(ROOT, "examples", "mxfp4_linear.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    first, last, W, x = ex.train(steps=60)
    # W starts at zero, so the first loss is the target's mean square, 1 within a
    # few percent; e2m1 inputs and weights carry noise of about 1 % of it each
    assert 0.9 < first < 1.1 and last < 0.15 * first
    # the three ways of one product differ by the order of fp32 sums and one bf16
    # step, 2^-8 of an entry
    assert ex.serve(W, x) <= 2.0 ** -8
