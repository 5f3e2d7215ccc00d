"""The Python functions of hkg_linear.h with tensors on a GPU that is not the current one,
and on two GPUs (CPU: stand-ins, as in test_ops_devices.py)."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_fp8_amd as hkg  # noqa: E402

from test_ops_devices import On, Stream, bf16, calls  # noqa: E402,F401


def every_call(a, b=None, **kw):
    """name -> call with its first tensor on GPU a, the others on b (default a)."""
    b = a if b is None else b
    bias = On(b, torch.zeros(16))
    rng = On(b, torch.zeros(2, dtype=torch.int64))
    return {
        "hkg_dropout": lambda: hkg.dropout(bf16(a, 64, 16), 0.5, rng, residual=bf16(b, 64, 16), **kw),
        "hkg_linear": lambda: hkg.linear(bf16(a, 64, 64), bf16(b, 16, 64), bias=bias, residual=bf16(b, 64, 16), p=0.5, rng=rng,
                                         z=bf16(b, 64, 16), **kw),
        "hkg_linear_backward": lambda: hkg.linear_backward(bf16(a, 64, 16), bf16(b, 64, 64), bf16(b, 16, 64), z=bf16(b, 64, 16),
                                                           activation="gelu", p=0.5, rng=rng, **kw),
    }


NAMES = list(every_call(0))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dev", [0, 1])
def test_runs_with_its_tensors_device_current(calls, name, dev):  # noqa: F811
    every_call(dev)[name]()
    assert calls == [(name, dev, 0)]
    assert torch.cuda.current_device() == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_belongs_to_the_tensors_device(calls, name):  # noqa: F811
    every_call(1, stream=Stream(1, 77))[name]()
    assert calls == [(name, 1, 77)]
    with pytest.raises(ValueError):
        every_call(1, stream=Stream(0, 78))[name]()
    assert len(calls) == 1


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_two_devices_are_refused(calls, name):  # noqa: F811
    with pytest.raises(ValueError):
        every_call(0, 1)[name]()
    assert calls == []


def test_only_the_generators_tensor_elsewhere_is_refused(calls):  # noqa: F811
    with pytest.raises(ValueError):
        hkg.dropout(bf16(0, 4, 4), 0.5, On(1, torch.zeros(2, dtype=torch.int64)))
    assert calls == []
