"""The layers between the linear ones: activations and gated activations, norms,
and the join of a block's output with its residual and the next block's norm,
each one kernel a direction.  All the arithmetic runs in the HIP library (see
capi and include/shampoo.h).

    u = norm(h, Norm("rms", w0))                          # before the first block
    y = train_linear(gated(train_linear(u, w_up), act="silu", keep="mx8"), w_down)
    h, u = join(h, y, after=Norm("rms", w1), gate=g, before=Norm("rms", w2), keep="mx8")

keep says what waits for the backward pass: "same", the inputs as they are, or
"mx8", copies of them in 8 bits (1.03 bytes an element, see mx8), from which
backward computes; outputs and row statistics are those of the inputs
themselves.  Arithmetic is fp32, rounded once into each output.  Calls run on
the current stream; tensors are float32 or bfloat16 on one device, of any
strides (rows that are not evenly spaced are copied first).  Gradients of gradients,
forward-mode tangents, torch.func's transforms and traces (torch.jit.trace,
make_fx) are refused; torch.compile runs the calls between its graphs.
"""
from __future__ import annotations

import math

import torch
from torch.autograd import forward_ad

from . import capi
from .mx4 import _has_tangent

_ACTS = {"silu": capi.ACT_SILU, "gelu": capi.ACT_GELU, "gelu_tanh": capi.ACT_GELU_TANH, "relu": capi.ACT_RELU,
         "relu2": capi.ACT_RELU2}
_KINDS = {"rms": capi.NORM_RMS, "layer": capi.NORM_LAYER}
_KEEP = {"same": False, "mx8": True}


def _low(keep):
    low = _KEEP.get(keep)
    if low is None:
        raise ValueError(f"keep must be one of {sorted(_KEEP)}")
    return low


def _refuse_tangents(*tensors):
    if any(t is not None and _has_tangent(t) for t in tensors):
        raise NotImplementedError("the layers form no tangents (no jvp)")


# ---------------------------------------------------------------------------
# Activations
# ---------------------------------------------------------------------------

def _activate(x, b, packed, act, keep):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    if forward_ad._current_level >= 0:
        _refuse_tangents(x, b)
    return capi.load_layers().activate(x, b, packed, code, _low(keep))


def activation(x, act="silu", keep="same"):
    """f(x) for act "silu", "gelu", "gelu_tanh", "relu" or "relu2" (the square of relu)."""
    return _activate(x, None, False, act, keep)


def gated(x, b=None, act="silu", keep="same"):
    """f(x) b.  Without b, x [..., 2 F] holds both: f of its first F columns times the
    other F, and its gradient is one matrix again."""
    return _activate(x, b, b is None, act, keep)


# ---------------------------------------------------------------------------
# Norms and joins
# ---------------------------------------------------------------------------

def _number(value, name):
    """value; a tensor that requires a gradient would get none, and is refused."""
    if isinstance(value, torch.Tensor) and value.requires_grad:
        raise ValueError(f"{name} is a number: no gradient of it is formed")
    return value


class Norm:
    """A norm over the last dimension: "rms", x / sqrt(mean(x^2) + eps), or
    "layer", (x - mean) / sqrt(variance + eps); times weight, plus bias
    (vectors, float32 or bfloat16; None: 1 and 0)."""

    __slots__ = ("weight", "bias", "_kind", "_code", "_eps")

    def __init__(self, kind="rms", weight=None, bias=None, eps=1e-6):
        self.kind, self.weight, self.bias, self.eps = kind, weight, bias, eps

    @property
    def kind(self):
        return self._kind

    @kind.setter
    def kind(self, kind):
        code = _KINDS.get(kind)
        if code is None:
            raise ValueError(f"kind must be one of {sorted(_KINDS)}")
        self._kind, self._code = kind, code

    @property
    def eps(self):
        return self._eps

    @eps.setter
    def eps(self, eps):
        if not 0.0 < _number(eps, "eps") < math.inf:
            raise ValueError("eps must be positive")
        self._eps = float(eps)


_NO_NORM = (capi.NORM_NONE, 0.0, None, None)


def _parts(n, name):
    if n is None:
        return _NO_NORM
    if not isinstance(n, Norm):
        raise ValueError(f"{name} must be a Norm")
    return n._code, n._eps, n.weight, n.bias


def norm(x, n, dtype=None, keep="same"):
    """The Norm n of x's rows, in `dtype` (x's own, or bfloat16 of a float32 x)."""
    kind, eps, w, b = _parts(n, "n")
    if kind == capi.NORM_NONE:
        raise ValueError("n must be a Norm")
    if dtype is not None and dtype is not x.dtype and not (x.dtype is torch.float32 and dtype is torch.bfloat16):
        raise ValueError(f"dtype {dtype} of a norm of {x.dtype}")
    if forward_ad._current_level >= 0:
        _refuse_tangents(x, w, b)
    return capi.load_layers().join(x, None, *_NO_NORM, None, 1.0, kind, eps, w, b, dtype is torch.bfloat16, _low(keep))[1]


def join(residual, branch, after=None, gate=None, scale=1.0, before=None, keep="same"):
    """(h, u) with h = scale residual + gate after(branch) and u = before(h).

    residual, branch  [..., C]; a float32 residual takes a bfloat16 branch too.
                  h has the residual's type, u the branch's
    after, before the Norm of the branch (None: the branch as it is) and the
                  next block's Norm (None: u is None)
    gate          [C]; [..., 1], a number for each row; or a row of C for each run of
                  the rows, such as [B, 1, C] for [B, S, C].  The backward pass sums
                  gradients of the gate, and of after's parameters, run by run, in
                  workspace of 4 bytes an element of the gate (8 where after has a bias):
                  with a row of the gate for each row that is as much as an fp32 h
    scale         a number"""
    if branch is None:
        raise ValueError("branch must be a tensor")
    n1, n2 = _parts(after, "after"), _parts(before, "before")
    if forward_ad._current_level >= 0:
        _refuse_tangents(residual, branch, gate, *n1[2:], *n2[2:])
    return capi.load_layers().join(residual, branch, *n1, gate, _number(scale, "scale"), *n2, False, _low(keep))
