"""Which device the layers' calls launch on when their tensors are not on the
current one, forward and backward; device and library are stand-ins (CPU)."""
import types

import pytest
import torch

import test_operators_device as D
from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from inverse_root_preconditioning_amd import mx8 as M8

machine = D.machine


class Tensor(D.Tensor):
    """As much of a tensor on cuda:`index` as the layers look at."""

    def contiguous(self):
        return self

    def element_size(self):
        return 4

    def new_empty(self, shape, dtype=None):
        return Tensor(shape if isinstance(shape, tuple) else (shape,), dtype or self.dtype, self.device.index)


@pytest.fixture
def layers(machine, monkeypatch):
    for mod in (L, M8):
        monkeypatch.setattr(mod, "_raw_stream", lambda index: ("stream of", index))
        monkeypatch.setattr(mod, "_current_device", lambda: machine.current)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(shape, dtype, device.index))
    monkeypatch.setattr(L, "_has_tangent", lambda t: False)
    return machine


def _x():
    return Tensor((8, 64))


def _norm():
    return L.Norm("rms", Tensor((64,)))


def _act_backward():
    ctx = types.SimpleNamespace(needs_input_grad=(True, False), low=False, saved_tensors=(_x(), None), packed=False,
                                gated=False, code=0, shape=torch.Size((8, 64)))
    return L._Activation.backward(ctx, _x())


def _join_backward():
    w = Tensor((64,))
    spec = L._Spec(_x(), _x(), _norm(), w, 1.0, _norm(), torch.float32, False)
    ctx = types.SimpleNamespace(spec=spec, types=(torch.float32, torch.float32),
                                needs_input_grad=(True, True, True, False, True, True, False, False),
                                saved_tensors=(_x(), _x(), w, None, w, w, None, None, Tensor((16, 2))))
    return L._Join.backward(ctx, _x(), _x())


CALLS = {
    "quantize": lambda: M8.quantize(_x()),
    "dequantize": lambda: M8.dequantize(M8.MX8Matrix.empty(8, 64, _x())),
    "activation": lambda: L.activation(_x()),
    "gated": lambda: L.gated(_x()),
    "gated of two": lambda: L.gated(_x(), _x()),
    "norm": lambda: L.norm(_x(), _norm()),
    "join": lambda: L.join(_x(), _x(), _norm(), Tensor((64,)), 1.0, _norm()),
    "activation backward": _act_backward,
    "join backward": _join_backward,
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device_is_current_at_the_launch(name, layers):
    CALLS[name]()
    assert layers.calls and all((dev, s) == (1, ("stream of", 1)) for _, dev, s in layers.calls)
    assert layers.current == 0


@pytest.mark.parametrize("call", [M8.quantize, lambda x, stream: M8.dequantize(M8.MX8Matrix.empty(8, 64, x), stream=stream)])
def test_a_stream_is_on_the_tensors_device_and_noted(call, layers):
    x = _x()
    stream = types.SimpleNamespace(device_index=1, cuda_stream=7)
    call(x, stream=stream)
    assert [(dev, s) for _, dev, s in layers.calls] == [(1, ("stream of", 1))]
    layers.calls.clear()
    with pytest.raises(ValueError, match="stream"):
        call(x, stream=types.SimpleNamespace(device_index=0, cuda_stream=7))
    assert not layers.calls
    M8.quantize(x, stream=stream)
    assert x.used_on is stream


def test_parameters_are_on_the_same_device(layers):
    other = Tensor((64,), index=0)
    for bad in (lambda: L.norm(_x(), L.Norm("rms", other)), lambda: L.norm(_x(), L.Norm("rms", Tensor((64,)), other)),
                lambda: L.join(_x(), _x(), gate=other), lambda: L.join(_x(), Tensor((8, 64), index=0)),
                lambda: L.gated(_x(), Tensor((8, 64), index=0))):
        with pytest.raises(ValueError, match="device|cuda:1"):
            bad()
    assert not layers.calls
