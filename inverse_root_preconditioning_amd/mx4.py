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
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import capi
from .adamw import _TYPES, _current_device, _on_stream, _raw_stream


def _padded(k):
    return (k + 127) & -128          # capi.MX4_PAD


_check = capi.check


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
        n = rows * _padded(cols) // 2             # a multiple of 64
        return cls._over(like.new_empty((n + n // 16,), dtype=torch.uint8), rows, cols)

    @classmethod
    def _over(cls, buf, rows, cols):
        """The matrix in a buffer of empty's layout."""
        m = cls.__new__(cls)
        n = rows * _padded(cols) // 2
        m._buf = buf
        m._codes = m._scales = None
        m.codes_ptr = m._buf.data_ptr()
        m.scales_ptr = m.codes_ptr + n
        m.rows, m.cols, m.device = rows, cols, buf.device
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

    def record_stream(self, stream):
        """As torch.Tensor.record_stream."""
        for t in (self._codes, self._scales) if self._buf is None else (self._buf,):
            t.record_stream(stream)


def _quantize(x, along_rows, along_cols):
    if x.dim() == 2 and x.stride(1) != 1 and x.stride(0) == 1 and x.shape[1] > 1:
        qt, q = _quantize(x.t(), along_cols, along_rows)
        return q, qt
    dtype, ld = _matrix(x, "x")
    index = x.device.index
    if index != _current_device():
        with torch.cuda.device(index):
            return _quantize(x, along_rows, along_cols)
    rows, cols = x.shape
    q = qt = None
    codes = scales = codes_t = scales_t = 0
    if along_rows:
        q = MX4Matrix.empty(rows, cols, x)
        codes, scales = q.codes_ptr, q.scales_ptr
    if along_cols:
        qt = MX4Matrix.empty(cols, rows, x)
        codes_t, scales_t = qt.codes_ptr, qt.scales_ptr
    rc = capi.load().shampoo_mx4_quantize(x.data_ptr(), dtype, rows, cols, ld, codes, scales, codes_t, scales_t,
                                          _raw_stream(index))
    if rc:
        _check(rc, "shampoo_mx4_quantize")
    return q, qt


def quantize(x, stream=None):
    """x [rows, cols] (or a transposed view of such a matrix) as MX4, 32
    consecutive columns sharing a scale."""
    if stream is not None:
        return _on_stream(stream, x.device, lambda: quantize(x), x)
    return _quantize(x, True, False)[0]


def quantize_both(x, stream=None):
    """(quantize(x), quantize(x.t())) from one reading of x."""
    if stream is not None:
        return _on_stream(stream, x.device, lambda: quantize_both(x), x)
    return _quantize(x, True, True)


def dequantize(q, dtype=torch.float32, stream=None):
    """The values of q."""
    if stream is not None:
        return _on_stream(stream, q.device, lambda: dequantize(q, dtype), q)
    code = _TYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be float32 or bfloat16")
    rows, cols, device = q.rows, q.cols, q.device
    if device.index != _current_device():
        with torch.cuda.device(device):
            return dequantize(q, dtype)
    out = torch.empty((rows, cols), dtype=dtype, device=device)
    rc = capi.load().shampoo_mx4_dequantize(q.codes_ptr, q.scales_ptr, rows, cols, out.data_ptr(), code, cols,
                                            _raw_stream(device.index))
    if rc:
        _check(rc, "shampoo_mx4_dequantize")
    return out


def _workspace(need, like):
    """Scratch memory (kept alive by the caller's frame) and its address."""
    if need == 0:
        return None, 0
    ws = like.new_empty(need, dtype=torch.uint8)
    return ws, ws.data_ptr()


def _refuse_gradient(t, name, call):
    """A product of raw memory has no graph: a gradient that it would cut is an error."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{call} forms no gradient of {name}: use train_linear, detach it, or call under no_grad")


def _has_tangent(t):
    # outside a dual level (the only case whose time counts) there are no tangents
    return forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None


def product(a, b, out=None, dtype=torch.bfloat16, alpha=1.0, beta=0.0, stream=None):
    """alpha a b^T + beta out, accumulated in fp32: a [M, K], b [N, K] -> [M, N].
    Written to `out` if given (of its type), else to a new matrix of `dtype`."""
    if stream is not None:
        return _on_stream(stream, a.device, lambda: product(a, b, out, dtype, alpha, beta), a, b, out)
    M, N, K, device = a.rows, b.rows, a.cols, a.device
    if K != b.cols:
        raise ValueError(f"a has {K} columns, b {b.cols}")
    if device != b.device or (out is not None and out.device != device):
        raise ValueError("the operands are on one device")
    if device.index != _current_device():
        with torch.cuda.device(device):
            return product(a, b, out, dtype, alpha, beta)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        if dtype not in _TYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        out = torch.empty((M, N), dtype=dtype, device=device)
    else:
        _refuse_gradient(out, "out", "product")
    ctype, ld = _matrix(out, "out")
    if out.shape != (M, N):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, N)}")
    lib = capi.load()
    need = lib.shampoo_mx4_workspace_bytes(M, N, K)
    ws, ws_ptr = _workspace(need, out)
    rc = lib.shampoo_mx4_product(a.codes_ptr, a.scales_ptr, b.codes_ptr, b.scales_ptr, M, N, K, alpha, beta,
                                 out.data_ptr(), ctype, ld, ws_ptr, need, _raw_stream(device.index))
    if rc:
        _check(rc, "shampoo_mx4_product")
    return out


def linear(x, w, out=None, stream=None):
    """mx4(x) w^T for x [..., K] and an MX4 weight w [N, K], in x's type.  It
    forms no gradients, and refuses an x that would need one."""
    if stream is not None:
        return _on_stream(stream, w.device, lambda: linear(x, w, out), x, w, out)
    shape, N, K, device = x.shape, w.rows, w.cols, w.device
    if shape[-1] != K:
        raise ValueError(f"x has {shape[-1]} columns, w {K}")
    if x.requires_grad:
        _refuse_gradient(x, "x", "linear")
    if _has_tangent(x):
        raise ValueError("linear forms no tangent of x")
    if x.device != device or (out is not None and out.device != device):
        raise ValueError("the operands are on one device")
    if device.index != _current_device():
        with torch.cuda.device(device):
            return linear(x, w, out)
    if len(shape) == 2:
        flat, rows, to = x, shape[0], (shape[0], N)
    else:
        rows, to = math.prod(shape[:-1]), (*shape[:-1], N)
        flat = x.view(rows, K)
    xtype, ldx = _matrix(flat, "x")
    ldy = N
    if out is None:
        out = x.new_empty(to)
    else:
        _refuse_gradient(out, "out", "linear")
        if out.shape != to or out.dtype != x.dtype:
            raise ValueError(f"out must have shape {to} and x's type")
        _, ldy = _matrix(out if len(to) == 2 else out.view(rows, N), "out")
    lib = capi.load()
    need = lib.shampoo_mx4_linear_workspace_bytes(rows, N, K)
    ws, ws_ptr = _workspace(need, x)
    rc = lib.shampoo_mx4_linear(flat.data_ptr(), ldx, w.codes_ptr, w.scales_ptr, rows, N, K, out.data_ptr(), ldy,
                                xtype, ws_ptr, need, _raw_stream(device.index))
    if rc:
        _check(rc, "shampoo_mx4_linear")
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
        # saved as tensors, so that backward frees them and hooks (offload, checkpoints) see them
        ctx.save_for_backward(xt._buf if need_w else None, wt._buf if need_x else None)
        ctx.types = x.dtype, w.dtype
        ctx.shape, ctx.w_shape, ctx.rows = x.shape, w.shape, flat.shape[0]
        return product(xq, wq, dtype=x.dtype).view(*x.shape[:-1], w.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad
        x_buf, w_buf = ctx.saved_tensors
        N, K = ctx.w_shape
        q, qt = _quantize(_flat(dy), need_x, need_w)
        dx = dw = None
        if need_x:
            dx = product(q, MX4Matrix._over(w_buf, K, N), dtype=ctx.types[0]).view(ctx.shape)
        if need_w:
            dw = product(qt, MX4Matrix._over(x_buf, K, ctx.rows), dtype=ctx.types[1])
        return dx, dw


def train_linear(x, w):
    """y = mx4(x) mx4(w)^T for x [..., K] and w [N, K], in x's type, with
    gradients through the quantisers as if they were the identity:
    dx = mx4(dy) mx4(w^T)^T and dw = mx4(dy^T) mx4(x^T)^T, every operand
    quantised along the dimension it is summed over.  What the backward pass
    needs is kept in MX4 (0.53 bytes an element).  Forward-mode tangents are refused."""
    if x.shape[-1] != w.shape[-1] or w.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} do not multiply")
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad) or _has_tangent(x) or _has_tangent(w):
        return _TrainLinear.apply(x, w)
    return product(quantize(_flat(x)), quantize(w.detach()), dtype=x.dtype).view(*x.shape[:-1], w.shape[0])
