"""Which device a call launches on when its tensors are not on the current one:
the library's stream handle 0 means the current device's, so the calls have to
make the tensors' device current.  Device and library are stand-ins (CPU)."""
import contextlib
import types

import pytest
import torch

from inverse_root_preconditioning_amd import adamw as AW
from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx4 as MX


class Tensor:
    """As much of a tensor on cuda:`index` as the calls look at."""
    requires_grad, is_cuda = False, True

    def __init__(self, shape, dtype=torch.float32, index=1):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def stride(self, i=None):
        s = (self.shape[1], 1) if self.dim() == 2 else (1,)
        return s if i is None else s[i]

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        self.used_on = stream

    def new_empty(self, shape, dtype=None):
        return Tensor(shape if isinstance(shape, tuple) else (shape,), dtype or self.dtype, self.device.index)


@pytest.fixture
def machine(monkeypatch):
    """Current device 0; records (device current at the call, stream) of every library call."""
    m = types.SimpleNamespace(current=0, calls=[])

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *a: 64

            def call(*args):
                m.calls.append((name, m.current, args[-1]))
                return 0
            return call

    @contextlib.contextmanager
    def enter(device):
        index = getattr(device, "index", device)
        was, m.current = m.current, index
        yield
        m.current = was

    lib = Lib()
    monkeypatch.setattr(capi, "load", lambda path=None: lib)
    for mod in (AW, MX):
        monkeypatch.setattr(mod, "_raw_stream", lambda index: ("stream of", index))
        monkeypatch.setattr(mod, "_current_device", lambda: m.current, raising=False)
    monkeypatch.setattr(torch.cuda, "device", enter)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: enter(s.device_index))
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(shape, dtype, device.index))
    monkeypatch.setattr(torch, "empty_like", lambda t, dtype=None: Tensor(t.shape, dtype, t.device.index))
    return m


def _table(index=1, layouts=(64,)):
    t = AW.TensorTable.__new__(AW.TensorTable)
    t.device, t.index, t.layouts = torch.device("cuda", index), index, layouts
    t.ptr = t.segments_ptr = 0x10000
    t.nsegments, t.type, t.n, t._norm_ws = 1, capi.T_F32, 1, 64
    t.tensor, t.segments, t._keep, t._streams = Tensor((1, 3), torch.int64, index), Tensor((1, 2)), [Tensor((64,))], set()
    return t


def _adamw(index=1):
    o = AW.AdamW.__new__(AW.AdamW)
    o.params, o._checked, o.t, o.seed, o.lr, o.betas, o.eps = _table(index), None, 0, 0, 1e-3, (0.9, 0.95), 1e-8
    o._copies_ptr = o._hyper_ptr = 0
    o.copies, o.hyper = None, Tensor((1, 2), index=index)
    o._state, o._state_ptrs = capi.STATE_MX8, (1, 2, 3, 4)
    o.m = o.v = o.m_scale = o.v_scale = Tensor((64,), torch.uint8, index)
    return o


def _matrix(index=1):
    return MX.MX4Matrix.empty(8, 64, Tensor((1,), index=index))


CALLS = {
    "grad_norm": lambda **k: AW.grad_norm(_table(), 1.0, **k),
    "step": lambda **k: _adamw().step(_table(), **k),
    "moments": lambda **k: _adamw().moments(**k),
    "quantize": lambda **k: MX.quantize(Tensor((8, 64)), **k),
    "quantize_both": lambda **k: MX.quantize_both(Tensor((8, 64)), **k),
    "dequantize": lambda **k: MX.dequantize(_matrix(), **k),
    "product": lambda **k: MX.product(_matrix(), _matrix(), **k),
    "linear": lambda **k: MX.linear(Tensor((8, 64)), _matrix(), **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device_is_current_at_the_launch(name, machine):
    CALLS[name]()
    assert machine.calls and all((dev, s) == (1, ("stream of", 1)) for _, dev, s in machine.calls)
    assert machine.current == 0


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_is_on_the_tensors_device(name, machine):
    stream = types.SimpleNamespace(device_index=1, cuda_stream=7)
    CALLS[name](stream=stream)
    assert machine.calls and all((dev, s) == (1, ("stream of", 1)) for _, dev, s in machine.calls)
    machine.calls.clear()
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](stream=types.SimpleNamespace(device_index=0, cuda_stream=7))
    assert not machine.calls


def test_small_operands_are_on_the_same_device(machine):
    one = Tensor((1,), index=0)
    with pytest.raises(ValueError, match="grad_scale"):
        _adamw().step(_table(), grad_scale=one)
    with pytest.raises(ValueError, match="out"):
        AW.grad_norm(_table(), 1.0, out=Tensor((2,), index=0))
    with pytest.raises(ValueError, match="device"):
        _adamw().step(_table(index=0))
    assert not machine.calls
    _adamw().step(_table(), grad_scale=Tensor((1,)))
    AW.grad_norm(_table(), 1.0, out=Tensor((2,)))
    assert len(machine.calls) == 2


def test_operands_of_another_stream_are_noted(machine):
    """The allocator learns of every operand that a call on `stream` uses."""
    s = types.SimpleNamespace(device_index=1, cuda_stream=7)
    x, q, r, out = Tensor((8, 64)), _matrix(), _matrix(), Tensor((8, 8))
    MX.quantize(x, stream=s)
    MX.dequantize(q, stream=s)
    MX.product(q, r, out=out, stream=s)
    table, opt, scale, norm = _table(), _adamw(), Tensor((1,)), Tensor((2,))
    AW.grad_norm(table, 1.0, out=norm, stream=s)
    opt.step(table, grad_scale=scale, stream=s)
    y, w = Tensor((8, 64)), _matrix()
    MX.linear(y, w, stream=s)
    used = [x, q._buf, r._buf, out, norm, scale, y, w._buf, table.tensor, table.segments, *table._keep, opt.hyper, opt.m,
            opt.params.tensor]
    assert all(t.used_on is s for t in used)
