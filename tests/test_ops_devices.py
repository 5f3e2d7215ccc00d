"""The Python functions of hkg_ops.h with tensors on a GPU that is not the current
one, and on two GPUs (CPU: tensors, torch's device functions and the library are
stand-ins that record what the calls see)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_fp8_amd as hkg  # noqa: E402
from dense_gemm_fp8_amd import ops  # noqa: E402


class On:
    """A CPU tensor that says it is on GPU `dev`."""
    is_cuda = True

    def __init__(self, dev, t):
        self.dev, self.t = dev, t

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    def __init__(self, dev, handle):
        self.device, self.cuda_stream = torch.device("cuda", dev), handle


@pytest.fixture
def calls(monkeypatch):
    """[(function, current device, stream handle)] of the launches; the current device is 0."""
    now, seen = [0], []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 0
                seen.append((name, now[0], args[-1]))
                return 0
            return call

    @contextlib.contextmanager
    def device(d):
        was, now[0] = now[0], d
        yield
        now[0] = was

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(ops, "_lib", lambda: Lib())
    monkeypatch.setattr(ops, "_raw_stream", lambda d: 0)        # every device's default stream
    monkeypatch.setattr(ops, "_several", True)
    return seen


def bf16(dev, *shape):
    return On(dev, torch.zeros(shape, dtype=torch.bfloat16))


def u8(dev, *shape):
    return On(dev, torch.zeros(shape, dtype=torch.uint8))


def every_call(a, b=None, **kw):
    """name -> call with its first tensor on GPU a, the others on b (default a)."""
    b = a if b is None else b
    s = u8(b, 512)
    return {
        "hkg_mxfp4_quantize": lambda: hkg.mxfp4_quantize(bf16(a, 64, 64), 0, **kw),
        "hkg_mxfp4_quantize_both": lambda: hkg.mxfp4_quantize_both(bf16(a, 64, 64), 0, 1, **kw),
        "hkg_mxfp4_dequantize": lambda: hkg.mxfp4_dequantize(u8(a, 64, 32), s, 0, **kw),
        "hkg_gemm_mxfp4": lambda: hkg.gemm_mxfp4(u8(a, 64, 32), u8(b, 64, 32), s, s, **kw),
        "hkg_linear_mxfp4": lambda: hkg.linear_mxfp4(bf16(a, 64, 64), u8(b, 64, 32), s, **kw),
        "hkg_linear_mxfp4_backward": lambda: hkg.linear_mxfp4_backward(bf16(a, 64, 64), u8(b, 64, 32), s, u8(b, 64, 32), s, **kw),
        "hkg_orthogonalize": lambda: hkg.orthogonalize(bf16(a, 64, 64), out=bf16(b, 64, 64), **kw),
    }


NAMES = list(every_call(0))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dev", [0, 1])
def test_runs_with_its_tensors_device_current(calls, name, dev):
    every_call(dev)[name]()
    assert calls == [(name, dev, 0)]
    assert torch.cuda.current_device() == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_belongs_to_the_tensors_device(calls, name):
    every_call(1, stream=Stream(1, 77))[name]()
    assert calls == [(name, 1, 77)]
    with pytest.raises(ValueError):
        every_call(1, stream=Stream(0, 78))[name]()
    assert len(calls) == 1


@pytest.mark.parametrize("name", [n for n in NAMES if "quantize" not in n or "de" in n])
def test_tensors_on_two_devices_are_refused(calls, name):
    with pytest.raises(ValueError):
        every_call(0, 1)[name]()
    assert calls == []


def test_keyword_arguments(calls):
    hkg.orthogonalize(G=bf16(1, 64, 64))
    assert calls == [("hkg_orthogonalize", 1, 0)]
    with pytest.raises(ValueError):
        hkg.orthogonalize(torch.zeros(4, 4))             # not a GPU tensor
