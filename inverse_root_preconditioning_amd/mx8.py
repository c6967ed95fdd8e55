"""8-bit microscaled (MX8) matrices: E4M3 values with one power-of-two scale for
32 consecutive columns, the form in which activations wait for the backward
pass (see layers, whose calls keep and read them by themselves).  All the
arithmetic runs in the HIP library (see capi and include/shampoo.h).

    q = quantize(x)                  # 1.03 bytes an element
    x = dequantize(q, x.dtype)       # within 2^-4 of each element, or 2^-17 of the largest of its 32
    with saved_tensors():            # what torch's own operations keep of bfloat16 inside is kept so
        y = block(x)
"""
from __future__ import annotations

import weakref

import torch
from torch.utils.weak import WeakTensorKeyDictionary

from . import capi
from .adamw import _TYPES, _current_device, _on_stream, _raw_stream
from .mx4 import _matrix

_MAX_COLS = 1 << 29                  # of a matrix of the library


def _padded(cols):
    return (cols + 31) & -32         # capi.GROUP


def _bytes(rows, cols):
    """Codes and scales of a matrix in one buffer, rounded up so that another may follow."""
    n = rows * _padded(cols)
    return (n + n // 32 + 15) & -16


class MX8Matrix:
    """A quantised matrix [rows, cols].  codes: uint8 [rows, padded], scales:
    uint8 [rows, padded / 32]; padded: cols rounded up to a multiple of 32."""

    __slots__ = ("_buf", "_codes", "_scales", "codes_ptr", "scales_ptr", "rows", "cols", "device")

    def __init__(self, codes, scales, rows, cols):
        k = _padded(cols)
        for name, t, width in (("codes", codes, k), ("scales", scales, k // capi.GROUP)):
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
        return cls._over(like.new_empty((_bytes(rows, cols),), dtype=torch.uint8), rows, cols)

    @classmethod
    def _over(cls, buf, rows, cols):
        """The matrix in a buffer of empty's layout."""
        m = cls.__new__(cls)
        m._buf = buf
        m._codes = m._scales = None
        m.codes_ptr = buf.data_ptr()
        m.scales_ptr = m.codes_ptr + rows * _padded(cols)
        m.rows, m.cols, m.device = rows, cols, buf.device
        return m

    @property
    def codes(self):
        if self._codes is None:
            k = _padded(self.cols)
            self._codes = self._buf[:self.rows * k].view(self.rows, k)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            n, k = self.rows * _padded(self.cols), _padded(self.cols) // capi.GROUP
            self._scales = self._buf[n:n + self.rows * k].view(self.rows, k)
        return self._scales

    @property
    def shape(self):
        return (self.rows, self.cols)

    def record_stream(self, stream):
        """As torch.Tensor.record_stream."""
        for t in (self._codes, self._scales) if self._buf is None else (self._buf,):
            t.record_stream(stream)


_tracing, _modes = torch._C._is_tracing, torch._C._len_torch_dispatch_stack   # cheap; the kind of a mode is not
_PROXY = torch._C._TorchDispatchModeKey.PROXY


def _in_trace():
    return _tracing() or torch._C._get_dispatch_mode(_PROXY) is not None


def _refuse_trace():
    """A trace would hold the allocation of the result and not the call that fills it."""
    if _in_trace():
        raise NotImplementedError("MX8 conversions cannot be recorded in a trace")


def quantize(x, stream=None):
    """x [rows, cols] as MX8, 32 consecutive columns sharing a scale; nearest even."""
    if _tracing() or _modes():
        _refuse_trace()
    if stream is not None:
        return _on_stream(stream, x.device, lambda: quantize(x), x)
    dtype, ld = _matrix(x, "x")
    if x.is_neg():                   # a view that negates what is in memory
        return quantize(x.resolve_neg())
    index = x.get_device()
    if index != _current_device():
        with torch.cuda.device(index):
            return quantize(x)
    rows, cols = x.shape
    q = MX8Matrix.empty(rows, cols, x)
    rc = capi.load().shampoo_mx8_quantize(x.data_ptr(), dtype, rows, cols, ld, q.codes_ptr, q.scales_ptr,
                                          _raw_stream(index))
    if rc:
        capi.check(rc, "shampoo_mx8_quantize")
    return q


def dequantize(q, dtype=torch.float32, stream=None):
    """The values of q."""
    if _tracing() or _modes():
        _refuse_trace()
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
    rc = capi.load().shampoo_mx8_dequantize(q.codes_ptr, q.scales_ptr, rows, cols, out.data_ptr(), code, cols,
                                            _raw_stream(device.index))
    if rc:
        capi.check(rc, "shampoo_mx8_dequantize")
    return out


# Of autograd's nodes those that hand their input on: copies of another type or layout, and views.
_COPIES = {"ToCopyBackward0", "CloneBackward0", "TBackward0", "TransposeBackward0", "PermuteBackward0", "ViewBackward0",
           "UnsafeViewBackward0", "ReshapeAliasBackward0", "AliasBackward0", "AsStridedBackward0", "SliceBackward0",
           "SelectBackward0", "SplitBackward0", "SplitWithSizesBackward0", "UnbindBackward0", "UnsqueezeBackward0",
           "SqueezeBackward0", "SqueezeBackward1", "ExpandBackward0"}


def _of_leaf(t):
    """Whether t is a leaf of autograd's graph, a view of one, or a copy of either."""
    node = t.grad_fn if t._base is None else t._base.grad_fn
    while node is not None and node.name() in _COPIES:
        node = node.next_functions[0][0]
    return node is None or node.name() == "torch::autograd::AccumulateGrad"


class _Kept:
    """A copy, alive while a graph that saved the tensor holds it."""

    __slots__ = ("q", "__weakref__")

    def __init__(self, q):
        self.q = q


def saved_tensors(min_elements=1 << 14, dtypes=(torch.bfloat16,)):
    """A context in which autograd keeps activations in MX8: every CUDA tensor of
    `dtypes` (bfloat16, float32) and at least `min_elements` that an operation
    inside saves for its backward pass and that autograd formed.  Backward then
    computes from the rounded values.

    Leaves stay as they are: parameters, trained or frozen, inputs, and what was formed
    without a gradient (masks, statistics); so do views of leaves and copies of
    them in another type, as mixed precision makes of its weights.  A weight that is
    computed otherwise (scaled, composed) is rounded like an activation: form
    it, and use it, outside.

    float32 is not rounded unless asked for, since operations on bfloat16 keep
    statistics in it (a norm's, the logarithms of an attention's sums) whose
    rounding would spoil their gradients.  For the same reason a loss belongs
    outside: what it keeps is a logarithm.  The operations of mx4 and layers keep
    integers, or with keep="same" their inputs, which are rounded like any others.
    Columns are the last dimension, with those before it where it is short.

    A tensor that several operations save has one copy, as it is one tensor to
    autograd: while a graph holds that copy and the tensor lives unchanged (autograd counts
    changes in place), on the same stream, and not while a graph is captured."""
    dtypes = tuple(dtypes)
    if not set(dtypes) <= set(_TYPES):
        raise ValueError("dtypes are of float32 and bfloat16")
    copies = WeakTensorKeyDictionary()   # tensor -> {version, part, layout and stream: its copy}, both weakly

    def copy_of(t, cols):
        def make():
            return _Kept(quantize(t.detach().reshape(-1, cols).contiguous()))
        if torch.cuda.is_current_stream_capturing():
            return make()
        layout = (t.numel(), cols) if t.is_contiguous() else (t.shape, t.stride())
        key = (t._version, t.dtype, t.is_neg(), t.storage_offset(), layout, _raw_stream(t.device.index))
        known = copies.setdefault(t if t._base is None else t._base, {})
        found = known.get(key)
        kept = found and found()
        if kept is None:
            for other, ref in list(known.items()):           # another thread may be here too
                if ref() is None:
                    known.pop(other, None)
            kept = make()
            known[key] = weakref.ref(kept)
        return kept

    def pack(t):
        if t.dtype not in dtypes or not t.is_cuda or t.numel() < max(min_elements, 1):
            return t
        if t.layout != torch.strided or _of_leaf(t) or _in_trace():
            return t
        # rows of less than two groups would be mostly padding; a vector is one row
        k, cols = t.dim(), 1
        while k and (k == t.dim() or cols < 2 * capi.GROUP and cols % capi.GROUP):
            k -= 1
            cols *= t.shape[k]
        if cols > _MAX_COLS:
            return t
        return copy_of(t, cols), t.dtype, t.shape

    def unpack(kept):
        if isinstance(kept, torch.Tensor):
            return kept
        copy, dtype, shape = kept
        return dequantize(copy.q, dtype).view(shape)
    return torch.autograd.graph.saved_tensors_hooks(pack, unpack)
