"""Calls of the layers and of mx8 inside a trace are refused (no GPU is used: they are refused first).  A
trace would record the allocation of their outputs and not what fills them."""
import pytest
import torch
from torch.fx.experimental.proxy_tensor import make_fx

from inverse_root_preconditioning_amd import layers as L
from inverse_root_preconditioning_amd import mx8 as M8

X = torch.zeros(4, 64)
CALLS = {"activation": lambda t: L.activation(t), "gated": lambda t: L.gated(t), "norm": lambda t: L.norm(t, L.Norm("rms")),
         "join": lambda t: L.join(t, t)[0], "quantize": lambda t: M8.dequantize(M8.quantize(t)),
         "dequantize": lambda t: M8.dequantize(None) + t}


@pytest.mark.parametrize("call", CALLS)
def test_jit_traces_are_refused(call):
    with pytest.raises(NotImplementedError, match="trace"):
        torch.jit.trace(CALLS[call], X, check_trace=False)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("mode", ["real", "fake", "symbolic"])
def test_fx_traces_are_refused(call, mode):
    with pytest.raises(NotImplementedError, match="trace"):
        make_fx(CALLS[call], tracing_mode=mode)(X)


@pytest.mark.parametrize("call", CALLS)
def test_outside_a_trace_what_is_wrong_is_the_tensor(call):
    with pytest.raises((ValueError, AttributeError)):
        CALLS[call](X)
