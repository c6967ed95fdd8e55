"""4-bit microscaled (MX4) matrices: E2M1 values with one power-of-two scale for
32 consecutive columns, their quantisation and their products on the scaled
MFMA.  All the arithmetic runs in the HIP library (see capi and
include/shampoo.h).

    wq = quantize(w)                 # once, for serving
    y = linear(x, wq)                # y = mx4(x) w^T, from one row to a whole prompt
    y = train_linear(x, w)           # the same with both gradients formed in MX4
"""
from __future__ import annotations

import math

import torch

from . import capi
from .adamw import _TYPES, _on_stream, _raw_stream


def _padded(k):
    return -(-k // capi.MX4_PAD) * capi.MX4_PAD


def _matrix(t, name):
    """t as (type, row stride); rows contiguous."""
    code = _TYPES.get(t.dtype)
    if code is None or not t.is_cuda:
        raise ValueError(f"{name} must be a float32 or bfloat16 CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    rows, cols = t.shape
    if t.is_contiguous():
        return code, cols
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        return code, cols
    if ld < cols:
        raise ValueError(f"the rows of {name} overlap")
    return code, ld


class MX4Matrix:
    """A quantised matrix [rows, cols].  codes: uint8 [rows, padded / 2], two
    values a byte; scales: uint8 [rows, padded / 32]; padded: cols rounded up
    to a multiple of 128."""

    __slots__ = ("_buf", "_codes", "_scales", "codes_ptr", "scales_ptr", "rows", "cols", "device")

    def __init__(self, codes, scales, rows, cols):
        k = _padded(cols)
        for name, t, width in (("codes", codes, k // 2), ("scales", scales, k // capi.GROUP)):
            if not (t.is_cuda and t.dtype == torch.uint8 and t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor")
            if tuple(t.shape) != (rows, width):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, width)}")
            if t.data_ptr() % 16:
                raise ValueError(f"{name} must be 16-byte aligned")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on one device")
        self._buf, self._codes, self._scales = None, codes, scales
        self.codes_ptr, self.scales_ptr = codes.data_ptr(), scales.data_ptr()
        self.rows, self.cols, self.device = rows, cols, codes.device

    @classmethod
    def empty(cls, rows, cols, like):
        """Uninitialised storage on the device of the tensor `like`: one buffer, scales after codes."""
        m = cls.__new__(cls)
        n = rows * _padded(cols) // 2             # a multiple of 64
        m._buf = like.new_empty(n + n // 16, dtype=torch.uint8)
        m._codes = m._scales = None
        m.codes_ptr = m._buf.data_ptr()
        m.scales_ptr = m.codes_ptr + n
        m.rows, m.cols, m.device = rows, cols, like.device
        return m

    @property
    def codes(self):
        if self._codes is None:
            n = self.rows * _padded(self.cols) // 2
            self._codes = self._buf[:n].view(self.rows, -1 if n else 0)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            n = self.rows * _padded(self.cols) // 2
            self._scales = self._buf[n:].view(self.rows, -1 if n else 0)
        return self._scales

    @property
    def shape(self):
        return (self.rows, self.cols)


def _quantize(x, along_rows, along_cols):
    if x.dim() == 2 and x.stride(1) != 1 and x.stride(0) == 1 and x.shape[1] > 1:
        qt, q = _quantize(x.t(), along_cols, along_rows)
        return q, qt
    dtype, ld = _matrix(x, "x")
    rows, cols = x.shape
    q = MX4Matrix.empty(rows, cols, x) if along_rows else None
    qt = MX4Matrix.empty(cols, rows, x) if along_cols else None
    capi.check(capi.shampoo_mx4_quantize(
        x.data_ptr(), dtype, rows, cols, ld, q.codes_ptr if q else 0, q.scales_ptr if q else 0,
        qt.codes_ptr if qt else 0, qt.scales_ptr if qt else 0, _raw_stream(x.device.index)), "shampoo_mx4_quantize")
    return q, qt


@_on_stream
def quantize(x):
    """x [rows, cols] (or a transposed view of such a matrix) as MX4, 32
    consecutive columns sharing a scale."""
    return _quantize(x, True, False)[0]


@_on_stream
def quantize_both(x):
    """(quantize(x), quantize(x.t())) from one reading of x."""
    return _quantize(x, True, True)


@_on_stream
def dequantize(q, dtype=torch.float32):
    """The values of q."""
    if dtype not in _TYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.device)
    capi.check(capi.shampoo_mx4_dequantize(q.codes_ptr, q.scales_ptr, q.rows, q.cols, out.data_ptr(), _TYPES[dtype],
                                           q.cols, _raw_stream(q.device.index)), "shampoo_mx4_dequantize")
    return out


def _workspace(need, like):
    """Scratch memory (kept alive by the caller's frame) and its address."""
    if need == 0:
        return None, 0
    ws = like.new_empty(need, dtype=torch.uint8)
    return ws, ws.data_ptr()


@_on_stream
def product(a, b, out=None, dtype=torch.bfloat16, alpha=1.0, beta=0.0):
    """alpha a b^T + beta out, accumulated in fp32: a [M, K], b [N, K] -> [M, N].
    Written to `out` if given (of its type), else to a new matrix of `dtype`."""
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    if a.device != b.device or (out is not None and out.device != a.device):
        raise ValueError("the operands are on one device")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        if dtype not in _TYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        out = torch.empty((a.rows, b.rows), dtype=dtype, device=a.device)
    ctype, ld = _matrix(out, "out")
    if tuple(out.shape) != (a.rows, b.rows):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(a.rows, b.rows)}")
    need = capi.shampoo_mx4_workspace_bytes(a.rows, b.rows, a.cols)
    ws, ws_ptr = _workspace(need, out)
    capi.check(capi.shampoo_mx4_product(a.codes_ptr, a.scales_ptr, b.codes_ptr, b.scales_ptr, a.rows, b.rows, a.cols,
                                        alpha, beta, out.data_ptr(), ctype, ld, ws_ptr, need,
                                        _raw_stream(a.device.index)), "shampoo_mx4_product")
    return out


@_on_stream
def linear(x, w, out=None):
    """mx4(x) w^T for x [..., K] and an MX4 weight w [N, K], in x's type."""
    shape = x.shape
    if shape[-1] != w.cols:
        raise ValueError(f"x has {shape[-1]} columns, w {w.cols}")
    if x.device != w.device or (out is not None and out.device != w.device):
        raise ValueError("the operands are on one device")
    rows = math.prod(shape[:-1])
    flat = x if len(shape) == 2 else x.view(rows, w.cols)
    xtype, ldx = _matrix(flat, "x")
    if out is None:
        out = x.new_empty((*shape[:-1], w.rows))
        ldy = w.rows
    else:
        if tuple(out.shape) != (*shape[:-1], w.rows) or out.dtype != x.dtype:
            raise ValueError(f"out must have shape {(*shape[:-1], w.rows)} and x's type")
        _, ldy = _matrix(out if out.dim() == 2 else out.view(rows, w.rows), "out")
    need = capi.shampoo_mx4_linear_workspace_bytes(rows, w.rows, w.cols)
    ws, ws_ptr = _workspace(need, x)
    capi.check(capi.shampoo_mx4_linear(flat.data_ptr(), ldx, w.codes_ptr, w.scales_ptr, rows, w.rows, w.cols,
                                       out.data_ptr(), ldy, xtype, ws_ptr, need, _raw_stream(x.device.index)),
               "shampoo_mx4_linear")
    return out


def _flat(t):
    return t.reshape(math.prod(t.shape[:-1]), t.shape[-1]).contiguous()


class _TrainLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        need_x, need_w = ctx.needs_input_grad
        flat = _flat(x.detach())
        xq, xt = _quantize(flat, True, need_w)
        wq, wt = _quantize(w.detach(), True, need_x)
        ctx.xt, ctx.wt = xt, wt
        ctx.types = x.dtype, w.dtype
        ctx.shape = x.shape
        return product(xq, wq, dtype=x.dtype).view(*x.shape[:-1], w.shape[0])

    @staticmethod
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad
        q, qt = _quantize(_flat(dy), need_x, need_w)
        dx = product(q, ctx.wt, dtype=ctx.types[0]).view(ctx.shape) if need_x else None
        dw = product(qt, ctx.xt, dtype=ctx.types[1]) if need_w else None
        return dx, dw


def train_linear(x, w):
    """y = mx4(x) mx4(w)^T for x [..., K] and w [N, K], in x's type, with
    gradients through the quantisers as if they were the identity:
    dx = mx4(dy) mx4(w^T)^T and dw = mx4(dy^T) mx4(x^T)^T, every operand
    quantised along the dimension it is summed over.  What the backward pass
    needs is kept in MX4 (0.53 bytes an element)."""
    if x.shape[-1] != w.shape[-1] or w.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} do not multiply")
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        return _TrainLinear.apply(x, w)
    return product(quantize(_flat(x)), quantize(w.detach()), dtype=x.dtype).view(*x.shape[:-1], w.shape[0])
