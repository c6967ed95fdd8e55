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
strides (rows that are not evenly spaced are copied first).  Gradients of gradients and
forward-mode tangents are refused.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import capi
from .adamw import _TYPES, _current_device, _raw_stream
from .mx4 import _has_tangent
from .mx8 import _bytes, _padded

_ACTS = {"silu": capi.ACT_SILU, "gelu": capi.ACT_GELU, "gelu_tanh": capi.ACT_GELU_TANH, "relu": capi.ACT_RELU,
         "relu2": capi.ACT_RELU2}
_KINDS = {"rms": capi.NORM_RMS, "layer": capi.NORM_LAYER}
_KEEP = {"same": False, "mx8": True}


def _low(keep):
    low = _KEEP.get(keep)
    if low is None:
        raise ValueError(f"keep must be one of {sorted(_KEEP)}")
    return low


def _type(t, name):
    code = _TYPES.get(t.dtype)
    if code is None or not t.is_cuda:
        raise ValueError(f"{name} must be a float32 or bfloat16 CUDA tensor")
    return code


def _rows(t):
    """(t, row stride) with evenly spaced rows of the last dimension: t itself or a copy."""
    if t.is_contiguous():
        return t, t.shape[-1]
    n = t.dim()
    if n > 1 and t.numel() and t.stride(-1) == 1 and t.stride(-2) >= t.shape[-1]:
        ld = t.stride(-2)
        for i in range(n - 2, 0, -1):
            if t.stride(i - 1) != t.stride(i) * t.shape[i]:
                break
        else:
            return t, ld
    return t.contiguous(), t.shape[-1]


def _differentiated(*tensors):
    """Whether a call has to go through autograd."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    for t in tensors:
        if t is not None and _has_tangent(t):
            return True
    return False


def _copies(buf, rows, cols, n):
    """Addresses of the codes and scales of n (of 2) MX8 matrices that lie one after the other in buf."""
    if buf is None:
        return 0, 0, 0, 0
    p, size, codes = buf.data_ptr(), _bytes(rows, cols), rows * _padded(cols)
    return (p, p + codes, p + size, p + size + codes) if n == 2 else (p, p + codes, 0, 0)


# ---------------------------------------------------------------------------
# Activations
# ---------------------------------------------------------------------------

def _act_forward(code, a, b, packed, low):
    """y and the MX8 copies (in one buffer; None unless `low`)."""
    index = a.device.index
    if index != _current_device():
        with torch.cuda.device(index):
            return _act_forward(code, a, b, packed, low)
    dtype = _type(a, "x")
    a, lda = _rows(a)
    width = a.shape[-1]
    cols = width // 2 if packed else width
    rows = a.numel() // width if width else 0
    y = a.new_empty(a.shape[:-1] + (cols,)) if packed else torch.empty(a.shape, dtype=a.dtype, device=a.device)
    pa = a.data_ptr()
    pb = ldb = 0
    if packed:
        pb, ldb = pa + cols * a.element_size(), lda
    elif b is not None:
        b, ldb = _rows(b)
        pb = b.data_ptr()
    n = 1 if not packed and b is None else 2
    buf = a.new_empty((n * _bytes(rows, cols),), dtype=torch.uint8) if low else None
    if rows and cols:
        rc = capi.load().shampoo_activation(code, pa, lda, pb, ldb, rows, cols, dtype, y.data_ptr(), cols,
                                            *_copies(buf, rows, cols, n), _raw_stream(index))
        if rc:
            capi.check(rc, "shampoo_activation")
    return y, buf


class _Activation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, b, packed, code, low):
        y, buf = _act_forward(code, a.detach(), None if b is None else b.detach(), packed, low)
        if low:
            ctx.save_for_backward(buf)
        else:
            ctx.save_for_backward(a, b)
        ctx.packed, ctx.code, ctx.low, ctx.shape, ctx.gated = packed, code, low, a.shape, packed or b is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        index = dy.device.index
        if index != _current_device():
            with torch.cuda.device(index):
                return _Activation.backward(ctx, dy)
        need_a, need_b = ctx.needs_input_grad[:2]
        da = torch.empty(ctx.shape, dtype=dy.dtype, device=dy.device) if need_a else None
        db = torch.empty(ctx.shape, dtype=dy.dtype, device=dy.device) if need_b else None
        if dy.numel() == 0:
            return da, db, None, None, None
        dy, lddy = _rows(dy)
        cols = dy.shape[-1]
        rows = dy.numel() // cols
        pa = lda = pb = ldb = 0
        kept = (0, 0, 0, 0)
        if ctx.low:
            buf, = ctx.saved_tensors
            kept = _copies(buf, rows, cols, 2 if ctx.gated else 1)
        else:
            a, b = ctx.saved_tensors
            a, lda = _rows(a)
            pa = a.data_ptr()
            if ctx.packed:
                pb, ldb = pa + cols * a.element_size(), lda
            elif b is not None:
                b, ldb = _rows(b)
                pb = b.data_ptr()
        pda, ldd = (da.data_ptr(), ctx.shape[-1]) if need_a else (0, 0)
        if ctx.packed:
            pdb, lddb = pda + cols * dy.element_size(), ldd
        else:
            pdb, lddb = (db.data_ptr(), cols) if need_b else (0, 0)
        rc = capi.load().shampoo_activation_backward(ctx.code, dy.data_ptr(), lddy, pa, lda, pb, ldb, *kept, ctx.gated,
                                                     rows, cols, _TYPES[dy.dtype], pda, ldd, pdb, lddb,
                                                     _raw_stream(index))
        if rc:
            capi.check(rc, "shampoo_activation_backward")
        return da, db, None, None, None


def _activate(a, b, packed, act, keep):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    low = _low(keep)
    _type(a, "x")
    if a.dim() == 0:
        raise ValueError("x must have a dimension")
    if _differentiated(a, b):
        return _Activation.apply(a, b, packed, code, low)
    return _act_forward(code, a, b, packed, False)[0]


def activation(x, act="silu", keep="same"):
    """f(x) for act "silu", "gelu", "gelu_tanh", "relu" or "relu2" (the square of relu)."""
    return _activate(x, None, False, act, keep)


def gated(x, b=None, act="silu", keep="same"):
    """f(x) b.  Without b, x [..., 2 F] holds both: f of its first F columns times the
    other F, and its gradient is one matrix again."""
    if b is None:
        if x.dim() and x.shape[-1] % 2:
            raise ValueError(f"x has {x.shape[-1]} columns: two halves are needed")
        return _activate(x, None, True, act, keep)
    if b.shape != x.shape or b.dtype != x.dtype or b.device != x.device:
        raise ValueError("x and b differ in shape, type or device")
    return _activate(x, b, False, act, keep)


# ---------------------------------------------------------------------------
# Norms and joins
# ---------------------------------------------------------------------------

class Norm:
    """A norm over the last dimension: "rms", x / sqrt(mean(x^2) + eps), or
    "layer", (x - mean) / sqrt(variance + eps); times weight, plus bias
    (vectors, float32 or bfloat16; None: 1 and 0)."""

    __slots__ = ("kind", "weight", "bias", "eps", "_code")

    def __init__(self, kind="rms", weight=None, bias=None, eps=1e-6):
        self._code = _KINDS.get(kind)
        if self._code is None:
            raise ValueError(f"kind must be one of {sorted(_KINDS)}")
        if not 0.0 < eps < math.inf:
            raise ValueError("eps must be positive")
        self.kind, self.weight, self.bias, self.eps = kind, weight, bias, float(eps)


def _vector(t, name, cols, device):
    """A vector of parameters: contiguous, with its address and type."""
    if t is None:
        return None, 0, 0
    code = _TYPES.get(t.dtype)
    if code is None or t.device != device:
        raise ValueError(f"{name} must be a float32 or bfloat16 tensor on {device}")
    if t.dim() != 1 or t.shape[0] != cols:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(cols,)}")
    t = t.contiguous()
    return t, t.data_ptr(), code


def _gate_rows(gate, shape):
    """(kind, rows that share a row of the gate) of a gate for rows of `shape`."""
    size, lead = gate.shape, shape[:-1]
    if size == shape[-1:]:
        return capi.GATE_ROWS, max(math.prod(lead), 1)
    if size == lead + (1,):
        return capi.GATE_TOKEN, 0
    # leading dimensions as they are, then ones, then the columns
    k = 0
    while k < len(lead) and k < len(size) and size[k] == lead[k]:
        k += 1
    if size != lead[:k] + (1,) * (len(lead) - k) + shape[-1:]:
        raise ValueError(f"gate has shape {tuple(size)}; expected {tuple(shape[-1:])}, {tuple(lead) + (1,)}, or one row "
                         f"of {shape[-1]} for each run of the rows of {tuple(shape)}")
    return capi.GATE_ROWS, max(math.prod(lead[k:]), 1)


class _Spec:
    """What a call says besides its tensors."""

    __slots__ = ("shape", "rows", "cols", "stream", "branch_dtype", "branch", "join", "scale", "kind1", "eps1", "kind2",
                 "eps2", "gate", "run", "low")

    def __init__(self, residual, branch, after, gate, scale, before, branch_dtype, low):
        self.shape = shape = residual.shape
        self.cols = shape[-1]
        self.rows = math.prod(shape[:-1])
        self.stream, self.branch_dtype, self.branch = _TYPES[residual.dtype], branch_dtype, _TYPES[branch_dtype]
        self.join, self.scale, self.low = branch is not None, scale, low
        self.kind1, self.eps1 = (0, 0.0) if after is None else (after._code, after.eps)
        self.kind2, self.eps2 = (0, 0.0) if before is None else (before._code, before.eps)
        self.gate, self.run = (capi.GATE_NONE, 0) if gate is None else _gate_rows(gate, shape)

    def keeps(self):
        """Which of residual and branch the backward pass reads."""
        return self.kind2 != 0, self.join and (self.kind1 != 0 or self.gate != 0 or self.kind2 != 0)

    def copies(self, buf):
        """Addresses of the codes and scales of residual and branch in their buffer."""
        out, at = [0, 0, 0, 0], 0
        if buf is not None:
            at, size, codes = buf.data_ptr(), _bytes(self.rows, self.cols), self.rows * _padded(self.cols)
            for i, kept in enumerate(self.keeps()):
                if kept:
                    out[2 * i:2 * i + 2] = at, at + codes
                    at += size
        return out

    def statistics(self, stats):
        """Addresses of the rows of mean and s of both norms in their tensor."""
        if stats is None:
            return 0, 0
        p = stats.data_ptr()
        first = p if self.kind1 else 0
        return first, (p + (8 * self.rows if self.kind1 else 0)) if self.kind2 else 0

    def pack(self, residual, branch, w1, b1, gate, w2, b2, buf, stats):
        """Bytes of a shampoo_join.  residual, branch: (address, row stride); the
        parameters: (tensor, address, type)."""
        return capi.JOIN.pack(self.rows, self.cols, self.stream, self.branch, *residual, *branch, self.scale,
                              self.kind1, self.eps1, *w1[1:], *b1[1:], self.kind2, self.eps2, *w2[1:], *b2[1:],
                              self.gate, *gate[1:], self.run, *self.copies(buf), *self.statistics(stats))


def _parameters(spec, w1, b1, gate, w2, b2, device):
    cols = spec.cols
    if gate is not None:
        code = _TYPES.get(gate.dtype)
        if code is None or gate.device != device:
            raise ValueError(f"gate must be a float32 or bfloat16 tensor on {device}")
        gate = gate.contiguous()
    return (_vector(w1, "after.weight", cols, device), _vector(b1, "after.bias", cols, device),
            (None, 0, 0) if gate is None else (gate, gate.data_ptr(), code),
            _vector(w2, "before.weight", cols, device), _vector(b2, "before.bias", cols, device))


def _join_forward(residual, branch, w1, b1, gate, w2, b2, spec, keep):
    """(h, u, MX8 copies, statistics), the last two for the backward pass with `keep`."""
    device = residual.device
    index = device.index
    if index != _current_device():
        with torch.cuda.device(index):
            return _join_forward(residual, branch, w1, b1, gate, w2, b2, spec, keep)
    parameters = _parameters(spec, w1, b1, gate, w2, b2, device)
    r, ldr = _rows(residual)
    y, ldy = _rows(branch) if spec.join else (None, 0)
    h = u = buf = stats = None
    if spec.join:
        h = torch.empty(spec.shape, dtype=residual.dtype, device=device)
    if spec.kind2:
        u = torch.empty(spec.shape, dtype=spec.branch_dtype, device=device)
    if keep:
        norms = (spec.kind1 != 0) + (spec.kind2 != 0)
        if norms:
            stats = r.new_empty((norms * spec.rows, 2), dtype=torch.float32)
        if spec.low:
            buf = r.new_empty((sum(spec.keeps()) * _bytes(spec.rows, spec.cols),), dtype=torch.uint8)
    if spec.rows and spec.cols:
        cols = spec.cols
        rc = capi.load().shampoo_join_forward(
            spec.pack((r.data_ptr(), ldr), (y.data_ptr(), ldy) if spec.join else (0, 0), *parameters, buf, stats),
            h.data_ptr() if spec.join else 0, cols, u.data_ptr() if spec.kind2 else 0, cols, _raw_stream(index))
        if rc:
            capi.check(rc, "shampoo_join_forward")
    return h, u, buf, stats


class _Join(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, branch, w1, b1, gate, w2, b2, spec):
        h, u, buf, stats = _join_forward(*(None if t is None else t.detach()
                                           for t in (residual, branch, w1, b1, gate, w2, b2)), spec, True)
        keep_r, keep_y = spec.keeps()
        if spec.low:
            keep_r = keep_y = False
        ctx.save_for_backward(residual if keep_r else None, branch if keep_y else None, w1, b1, gate, w2, b2, buf, stats)
        ctx.set_materialize_grads(False)
        ctx.spec, ctx.types = spec, (residual.dtype, spec.branch_dtype)
        return (h, u) if spec.join and spec.kind2 else h if spec.join else u

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        spec = ctx.spec
        given = next((g for g in grads if g is not None), None)
        if given is None:
            return (None,) * 8
        device = given.device
        index = device.index
        if index != _current_device():
            with torch.cuda.device(index):
                return _Join.backward(ctx, *grads)
        residual, branch, w1, b1, gate, w2, b2, buf, stats = ctx.saved_tensors
        dh = grads[0] if spec.join else None
        du = grads[-1] if spec.kind2 else None
        need = list(ctx.needs_input_grad[:7])
        if du is None:
            need[5] = need[6] = False
        shapes = (spec.shape, spec.shape, *(None if t is None else t.shape for t in (w1, b1, gate, w2, b2)))
        dtypes = (*ctx.types, *(None if t is None else t.dtype for t in (w1, b1, gate, w2, b2)))
        if not (spec.rows and spec.cols):
            return (*(torch.zeros(n, dtype=t, device=device) if k else None for k, n, t in zip(need, shapes, dtypes)), None)
        out = [torch.empty(n, dtype=t, device=device) if k else None for k, n, t in zip(need, shapes, dtypes)]
        ptr = [0 if t is None else t.data_ptr() for t in out]
        parameters = _parameters(spec, w1, b1, gate, w2, b2, device)
        dh, lddh = (None, 0) if dh is None else _rows(dh)
        du, lddu = (None, 0) if du is None else _rows(du)
        # where only the copies are read, an address that says there is such an input
        r, ldr = (None, spec.cols) if residual is None else _rows(residual)
        y, ldy = (None, spec.cols) if branch is None else _rows(branch)
        at = given.data_ptr()
        cols = spec.cols
        lib = capi.load()
        packed = spec.pack((at if r is None else r.data_ptr(), ldr),
                           ((at if y is None else y.data_ptr()) if spec.join else 0, ldy), *parameters, buf, stats)
        size = lib.shampoo_join_workspace_bytes(packed)
        ws = given.new_empty((size,), dtype=torch.uint8)
        rc = lib.shampoo_join_backward(
            packed, capi.JOIN_GRADS.pack(0 if dh is None else dh.data_ptr(), lddh, 0 if du is None else du.data_ptr(), lddu,
                                         ptr[0], cols, ptr[1], cols, *ptr[2:]),
            ws.data_ptr(), size, _raw_stream(index))
        if rc:
            capi.check(rc, "shampoo_join_backward")
        return (*out, None)


def _checked_norm(n, name):
    if n is not None and not isinstance(n, Norm):
        raise ValueError(f"{name} must be a Norm")
    return (None, None) if n is None else (n.weight, n.bias)


def norm(x, n, dtype=None, keep="same"):
    """The Norm n of x's rows, in `dtype` (x's own, or bfloat16 of a float32 x)."""
    low = _low(keep)
    if n is None:
        raise ValueError("n must be a Norm")
    w, b = _checked_norm(n, "n")
    _type(x, "x")
    dtype = x.dtype if dtype is None else dtype
    if dtype is not x.dtype and not (x.dtype is torch.float32 and dtype is torch.bfloat16):
        raise ValueError(f"dtype {dtype} of a norm of {x.dtype}")
    if x.dim() == 0:
        raise ValueError("x must have a dimension")
    spec = _Spec(x, None, None, None, 1.0, n, dtype, low)
    if _differentiated(x, w, b):
        return _Join.apply(x, None, None, None, None, w, b, spec)
    return _join_forward(x, None, None, None, None, w, b, spec, False)[1]


def join(residual, branch, after=None, gate=None, scale=1.0, before=None, keep="same"):
    """(h, u) with h = scale residual + gate after(branch) and u = before(h).

    residual, branch  [..., C]; a float32 residual takes a bfloat16 branch too.
                  h has the residual's type, u the branch's
    after, before the Norm of the branch (None: the branch as it is) and the
                  next block's Norm (None: u is None)
    gate          [C]; [..., 1], a number for each row; or a row of C for each run of
                  the rows, such as [B, 1, C] for [B, S, C]
    scale         a number"""
    low = _low(keep)
    w1, b1 = _checked_norm(after, "after")
    w2, b2 = _checked_norm(before, "before")
    _type(residual, "residual"), _type(branch, "branch")
    if branch.shape != residual.shape or branch.device != residual.device:
        raise ValueError("residual and branch differ in shape or device")
    if residual.dim() == 0:
        raise ValueError("residual must have a dimension")
    if branch.dtype is not residual.dtype and residual.dtype is not torch.float32:
        raise ValueError(f"a {branch.dtype} branch of a {residual.dtype} residual")
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    spec = _Spec(residual, branch, after, gate, scale, before, branch.dtype, low)
    if _differentiated(residual, branch, w1, b1, gate, w2, b2):
        out = _Join.apply(residual, branch, w1, b1, gate, w2, b2, spec)
        return out if spec.kind2 else (out, None)
    return _join_forward(residual, branch, w1, b1, gate, w2, b2, spec, False)[:2]
