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
from .adamw import _TYPES, _on


def _padded(k):
    return -(-k // capi.MX4_PAD) * capi.MX4_PAD


def _matrix(t, name):
    """t as (type, row stride); rows contiguous."""
    if not t.is_cuda or t.dtype not in _TYPES:
        raise ValueError(f"{name} must be a float32 or bfloat16 CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"the rows of {name} overlap")
    return _TYPES[t.dtype], ld


class MX4Matrix:
    """A quantised matrix [rows, cols].  codes: uint8 [rows, padded / 2], two
    values a byte; scales: uint8 [rows, padded / 32]; padded: cols rounded up
    to a multiple of 128."""

    __slots__ = ("codes", "scales", "rows", "cols")

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
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols

    @classmethod
    def empty(cls, rows, cols, device):
        """Uninitialised storage."""
        k = _padded(cols)
        m = cls.__new__(cls)
        m.codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=device)
        m.scales = torch.empty((rows, k // capi.GROUP), dtype=torch.uint8, device=device)
        m.rows, m.cols = rows, cols
        return m

    @property
    def device(self):
        return self.codes.device

    @property
    def shape(self):
        return (self.rows, self.cols)


def _quantize(x, along_rows, along_cols, stream):
    if x.dim() == 2 and x.stride(1) != 1 and x.stride(0) == 1 and x.shape[1] > 1:
        qt, q = _quantize(x.t(), along_cols, along_rows, stream)
        return q, qt
    dtype, ld = _matrix(x, "x")
    rows, cols = x.shape
    with _on(stream):
        q = MX4Matrix.empty(rows, cols, x.device) if along_rows else None
        qt = MX4Matrix.empty(cols, rows, x.device) if along_cols else None
        capi.check(capi.shampoo_mx4_quantize(
            x.data_ptr(), dtype, rows, cols, ld, q.codes.data_ptr() if q else 0, q.scales.data_ptr() if q else 0,
            qt.codes.data_ptr() if qt else 0, qt.scales.data_ptr() if qt else 0,
            torch.cuda.current_stream(x.device).cuda_stream), "shampoo_mx4_quantize")
    return q, qt


def quantize(x, stream=None):
    """x [rows, cols] (or a transposed view of such a matrix) as MX4, 32
    consecutive columns sharing a scale."""
    return _quantize(x, True, False, stream)[0]


def quantize_both(x, stream=None):
    """(quantize(x), quantize(x.t())) from one reading of x."""
    return _quantize(x, True, True, stream)


def dequantize(q, dtype=torch.float32, stream=None):
    """The values of q."""
    if dtype not in _TYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    with _on(stream):
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.device)
        capi.check(capi.shampoo_mx4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, out.data_ptr(),
                                               _TYPES[dtype], q.cols,
                                               torch.cuda.current_stream(out.device).cuda_stream),
                   "shampoo_mx4_dequantize")
    return out


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def product(a, b, out=None, dtype=torch.bfloat16, alpha=1.0, beta=0.0, stream=None):
    """alpha a b^T + beta out, accumulated in fp32: a [M, K], b [N, K] -> [M, N].
    Written to `out` if given (of its type), else to a new matrix of `dtype`."""
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    if a.device != b.device or (out is not None and out.device != a.device):
        raise ValueError("the operands are on one device")
    with _on(stream):
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
        ws = _workspace(need, a.device) if need else None
        capi.check(capi.shampoo_mx4_product(
            a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(), a.rows, b.rows, a.cols,
            alpha, beta, out.data_ptr(), ctype, ld, ws.data_ptr() if need else 0, need,
            torch.cuda.current_stream(a.device).cuda_stream), "shampoo_mx4_product")
    return out


def linear(x, w, out=None, stream=None):
    """mx4(x) w^T for x [..., K] and an MX4 weight w [N, K], in x's type."""
    if x.shape[-1] != w.cols:
        raise ValueError(f"x has {x.shape[-1]} columns, w {w.cols}")
    if x.device != w.device or (out is not None and out.device != w.device):
        raise ValueError("the operands are on one device")
    rows = math.prod(x.shape[:-1])
    flat = x if x.dim() == 2 else x.view(rows, w.cols)
    xtype, ldx = _matrix(flat, "x")
    with _on(stream):
        if out is None:
            out = torch.empty((*x.shape[:-1], w.rows), dtype=x.dtype, device=x.device)
        elif tuple(out.shape) != (*x.shape[:-1], w.rows) or out.dtype != x.dtype:
            raise ValueError(f"out must have shape {(*x.shape[:-1], w.rows)} and x's type")
        _, ldy = _matrix(out if out.dim() == 2 else out.view(rows, w.rows), "out")
        need = capi.shampoo_mx4_linear_workspace_bytes(rows, w.rows, w.cols)
        ws = _workspace(need, x.device)
        capi.check(capi.shampoo_mx4_linear(
            flat.data_ptr(), ldx, w.codes.data_ptr(), w.scales.data_ptr(), rows, w.rows, w.cols, out.data_ptr(), ldy,
            xtype, ws.data_ptr(), need, torch.cuda.current_stream(x.device).cuda_stream), "shampoo_mx4_linear")
    return out


def _flat(t):
    return t.reshape(math.prod(t.shape[:-1]), t.shape[-1]).contiguous()


class _TrainLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        need_x, need_w = ctx.needs_input_grad
        flat = _flat(x.detach())
        xq, xt = _quantize(flat, True, need_w, None)
        wq, wt = _quantize(w.detach(), True, need_x, None)
        ctx.xt, ctx.wt = xt, wt
        ctx.types = x.dtype, w.dtype
        ctx.shape = x.shape
        return product(xq, wq, dtype=x.dtype).view(*x.shape[:-1], w.shape[0])

    @staticmethod
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad
        q, qt = _quantize(_flat(dy), need_x, need_w, None)
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
