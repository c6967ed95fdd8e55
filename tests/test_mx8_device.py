"""Which device the MX8 calls launch on when their tensors are not on the
current one; device and library are stand-ins (CPU)."""
import types

import pytest
import torch

import test_operators_device as D
from inverse_root_preconditioning_amd import mx8 as M8

machine = D.machine


class Tensor(D.Tensor):
    """As much of a tensor on cuda:`index` as the calls look at."""

    def contiguous(self):
        return self

    def is_neg(self):
        return False

    def element_size(self):
        return 4

    def new_empty(self, shape, dtype=None):
        return Tensor(shape if isinstance(shape, tuple) else (shape,), dtype or self.dtype, self.device.index)


@pytest.fixture
def mx8(machine, monkeypatch):
    monkeypatch.setattr(M8, "_raw_stream", lambda index: ("stream of", index))
    monkeypatch.setattr(M8, "_current_device", lambda: machine.current)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(shape, dtype, device.index))
    return machine


def _x():
    return Tensor((8, 64))


CALLS = {
    "quantize": lambda: M8.quantize(_x()),
    "dequantize": lambda: M8.dequantize(M8.MX8Matrix.empty(8, 64, _x())),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device_is_current_at_the_launch(name, mx8):
    CALLS[name]()
    assert mx8.calls and all((dev, s) == (1, ("stream of", 1)) for _, dev, s in mx8.calls)
    assert mx8.current == 0


@pytest.mark.parametrize("call", [M8.quantize, lambda x, stream: M8.dequantize(M8.MX8Matrix.empty(8, 64, x), stream=stream)])
def test_a_stream_is_on_the_tensors_device_and_noted(call, mx8):
    x = _x()
    stream = types.SimpleNamespace(device_index=1, cuda_stream=7)
    call(x, stream=stream)
    assert [(dev, s) for _, dev, s in mx8.calls] == [(1, ("stream of", 1))]
    mx8.calls.clear()
    with pytest.raises(ValueError, match="stream"):
        call(x, stream=types.SimpleNamespace(device_index=0, cuda_stream=7))
    assert not mx8.calls
    M8.quantize(x, stream=stream)
    assert x.used_on is stream
