"""AdamW over many tensors at once, with its moments in 32 or in 8 bits, and
the norm that clips their gradients: the step for the tensors that the block
preconditioner leaves (norm vectors, biases, embeddings), or for all of them.
All the arithmetic runs in the HIP library (see capi and include/shampoo.h).

    grads = TensorTable([p.grad for p in params])
    opt = AdamW(params, lr=1e-3, weight_decay=0.1, state="mx8")
    norm = grad_norm(grads, 1.0)               # [norm, clipping factor], on the device
    opt.step(grads, grad_scale=norm[1:])
"""
from __future__ import annotations

import numpy as np
import torch

from . import capi

_TYPES = {torch.float32: capi.T_F32, torch.bfloat16: capi.T_BF16}
_STATES = {"f32": capi.STATE_F32, "mx8": capi.STATE_MX8}

_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream(i).cuda_stream without the Python objects
_current_device = torch._C._cuda_getDevice


def _on_stream(stream, device, call, *operands):
    """call() on `stream`; the operands (None: not given) are on `device`.  They
    may be another stream's memory and be freed there before the call has run, so
    the allocator is told of it."""
    if stream.device_index != device.index:
        raise ValueError(f"the stream is on device {stream.device_index}, the tensors on {device}")
    with torch.cuda.stream(stream):
        result = call()
    for t in operands:
        if t is not None:
            t.record_stream(stream)
    return result


def _dense(t):
    """Whether t fills one stretch of memory without gaps or overlap."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != want:
            return False
        want *= size
    return True


def _layout(t):
    """What two tensors must share for their flat orders to name the same elements."""
    if t.is_contiguous():
        return t.numel()
    # dimensions of one element are in no order
    return tuple(size for size in t.shape if size != 1), tuple(st for st, size in zip(t.stride(), t.shape) if size != 1)


def _nested_tuple(x):
    return tuple(map(_nested_tuple, x)) if isinstance(x, (list, tuple)) else x


class TensorTable:
    """Device table of tensors in their flat memory order (the tensors are kept
    alive with it).  All of one type, float32 or bfloat16, and dense.  A table
    is built again when its tensors move (gradients that are freed between
    steps); tensors whose memory stays need it once."""

    def __init__(self, tensors):
        tensors = list(tensors)
        dtypes = {t.dtype for t in tensors}
        if len(dtypes) > 1:
            raise ValueError("the tensors of a table have one type")
        dtype = dtypes.pop() if dtypes else torch.float32
        if dtype not in _TYPES:
            raise ValueError(f"tensors must be float32 or bfloat16, not {dtype}")
        for i, t in enumerate(tensors):
            if not t.is_cuda:
                raise ValueError(f"tensor {i} is not a CUDA tensor")
            if t.device != tensors[0].device:
                raise ValueError("the tensors of a table are on one device")
            if not _dense(t):
                raise ValueError(f"tensor {i} is not dense")
        self.dtype = dtype
        self.type = _TYPES[dtype]
        self.device = tensors[0].device if tensors else torch.device("cuda", torch.cuda.current_device())
        self.index = self.device.index
        self.layouts = tuple(_layout(t) for t in tensors)
        self._keep = tensors
        sizes = np.array([t.numel() for t in tensors], dtype=np.int64)
        padded = (sizes + capi.GROUP - 1) // capi.GROUP * capi.GROUP
        self.offsets = np.concatenate([np.zeros(1, np.int64), np.cumsum(padded)]).astype(np.int64)
        self.total = int(self.offsets[-1])   # elements of a state buffer
        self.sizes = sizes
        self.n = len(tensors)
        rows = np.zeros((max(self.n, 1), 3), dtype=np.int64)
        for i, t in enumerate(tensors):
            rows[i] = t.data_ptr(), sizes[i], self.offsets[i]
        pieces = (sizes + capi.SEGMENT - 1) // capi.SEGMENT
        if self.n and int(pieces.max()) > 0x7FFFFFFF:
            raise ValueError("a tensor is too large for the segment list")
        self.nsegments = int(pieces.sum())
        seg = np.zeros((max(self.nsegments, 1), 2), dtype=np.int32)
        seg[:self.nsegments, 0] = np.repeat(np.arange(self.n), pieces)
        seg[:self.nsegments, 1] = np.arange(self.nsegments) - np.repeat(np.cumsum(pieces) - pieces, pieces)
        self.tensor = torch.from_numpy(rows).to(self.device)
        self.segments = torch.from_numpy(seg).to(self.device)
        self.ptr = self.tensor.data_ptr()
        self.segments_ptr = self.segments.data_ptr()
        self._norm_ws = capi.shampoo_grad_norm_workspace_bytes(self.nsegments)
        self._streams = set()

    def record_stream(self, stream):
        """As torch.Tensor.record_stream, for the table and its tensors (a use is noted until they are freed)."""
        if stream.cuda_stream not in self._streams:
            for t in (self.tensor, self.segments, *self._keep):
                t.record_stream(stream)
            self._streams.add(stream.cuda_stream)


def grad_norm(table, max_norm=float("inf"), out=None, stream=None):
    """float32 [2] on the device: the Euclidean norm of all the table's tensors
    as one vector, and min(1, max_norm / norm) (NaN if the norm is not finite,
    which makes AdamW.step change nothing)."""
    if stream is not None:
        return _on_stream(stream, table.device, lambda: grad_norm(table, max_norm, out), table, out)
    if table.index != _current_device():
        with torch.cuda.device(table.index):
            return grad_norm(table, max_norm, out)
    if out is None:
        out = table.tensor.new_empty((2,), dtype=torch.float32)
    elif not (out.get_device() == table.index and out.dtype == torch.float32 and out.is_contiguous()
              and out.numel() == 2):
        raise ValueError("out must be a contiguous float32 CUDA tensor of 2 elements on the table's device")
    need = table._norm_ws
    ws = table.tensor.new_empty(need, dtype=torch.uint8) if need else None
    rc = capi.load().shampoo_grad_norm(table.ptr, table.segments_ptr, table.nsegments, table.type, max_norm,
                                       out.data_ptr(), ws.data_ptr() if need else 0, need, _raw_stream(table.index))
    if rc:
        capi.check(rc, "shampoo_grad_norm")
    return out


def _refuse_shared(tensors, name):
    """Two segments of a step must not update the same memory."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t.numel())
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        raise ValueError(f"{name} share memory")


def _per_tensor(value, n, name):
    values = [float(v) for v in value] if isinstance(value, (list, tuple)) else [float(value)] * n
    if len(values) != n:
        raise ValueError(f"{name} has {len(values)} values for {n} tensors")
    return values


class AdamW:
    """AdamW (decoupled weight decay) over a list of tensors, updated in place.

    params        float32 or bfloat16 tensors of one type, or a TensorTable, apart
                  from one another (a tied weight is given once).
                  bfloat16 parameters are rounded stochastically, so that steps
                  below their spacing are kept on average
    weight_decay  a number, or one for each tensor
    lr_scale      factor on the learning rate, a number or one for each tensor
    state         "f32", or "mx8": two bytes of moments an element
    copies        bfloat16 tensors that receive the float32 parameters, rounded
    seed          of the stochastic rounding: equal seeds give equal bits

    The moments live in flat buffers, every tensor starting at a multiple of
    32 elements (`offsets`).  `t` counts the steps taken; a step captured into a
    graph keeps its count, so that every replay repeats its bias correction and
    its random bits (whose rounding is then no longer unbiased over the steps),
    and `t` does not advance.  The parameters change outside autograd's sight:
    run a backward pass that needs their old values before the step."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, lr_scale=1.0, state="f32",
                 copies=None, seed=0):
        self.params = params if isinstance(params, TensorTable) else TensorTable(params)
        if state not in _STATES:
            raise ValueError(f"state must be one of {sorted(_STATES)}")
        b1, b2 = betas
        if not (0.0 <= b1 < 1.0 and 0.0 <= b2 < 1.0 and eps >= 0.0):
            raise ValueError("need 0 <= betas < 1 and eps >= 0")
        self.lr, self.betas, self.eps, self.seed, self.t = lr, (float(b1), float(b2)), eps, int(seed), 0
        if not 0 <= self.seed < 1 << 64:
            raise ValueError("seed must fit 64 bits")
        self.state = state
        p, dev = self.params, self.params.device
        self.offsets = p.offsets
        self.copies = self._checked = None
        if copies is not None:
            self.copies = copies if isinstance(copies, TensorTable) else TensorTable(copies)
            if p.dtype != torch.float32 or self.copies.dtype != torch.bfloat16:
                raise ValueError("copies are bfloat16 copies of float32 parameters")
            self._same(self.copies, "copies")
        _refuse_shared(p._keep + (self.copies._keep if self.copies else []), "parameters or copies")
        hyper = np.array([_per_tensor(lr_scale, p.n, "lr_scale"), _per_tensor(weight_decay, p.n, "weight_decay")],
                         dtype=np.float32).T
        self.hyper = torch.from_numpy(np.ascontiguousarray(hyper)).to(dev)
        low = state == "mx8"
        dtype = torch.uint8 if low else torch.float32
        self.m = torch.zeros(p.total, dtype=dtype, device=dev)
        self.v = torch.zeros(p.total, dtype=dtype, device=dev)
        self.m_scale = torch.zeros(p.total // capi.GROUP, dtype=torch.uint8, device=dev) if low else None
        self.v_scale = torch.zeros(p.total // capi.GROUP, dtype=torch.uint8, device=dev) if low else None
        # the buffers stay where they are: load_state_dict copies into them
        self._state = _STATES[state]
        self._state_ptrs = tuple(0 if t is None else t.data_ptr() for t in (self.m, self.v, self.m_scale, self.v_scale))
        self._hyper_ptr = self.hyper.data_ptr()
        self._copies_ptr = 0 if self.copies is None else self.copies.ptr

    def _same(self, table, name):
        if table.layouts != self.params.layouts:
            raise ValueError(f"{name} differ from the parameters in number, size or layout")
        if table.device != self.params.device:
            raise ValueError(f"{name} are on another device than the parameters")

    def record_stream(self, stream):
        """As torch.Tensor.record_stream, for the parameters, their copies and the state."""
        self.params.record_stream(stream)
        for t in (self.copies, self.hyper, self.m, self.v, self.m_scale, self.v_scale):
            if t is not None:
                t.record_stream(stream)

    def step(self, grads, lr=None, grad_scale=None, stream=None):
        """One step with the gradients of a TensorTable (or a list of tensors).
        grad_scale: float32 tensor of one element on the device that multiplies
        the gradients; if it is not finite, nothing changes but `t`."""
        p = self.params
        if stream is not None:
            grads = grads if isinstance(grads, TensorTable) else list(grads)
            return _on_stream(stream, p.device, lambda: self.step(grads, lr, grad_scale), self, grad_scale,
                              *((grads,) if isinstance(grads, TensorTable) else grads))
        if p.index != _current_device():
            with torch.cuda.device(p.index):
                return self.step(grads, lr, grad_scale)
        if not isinstance(grads, TensorTable):
            grads = TensorTable(grads)
        # Layouts found equal are found again by their tuple; the table itself, and the gradients with it, is not kept.
        if grads.layouts is not self._checked or grads.index != p.index:
            self._same(grads, "gradients")
            self._checked = grads.layouts
        scale_ptr = 0
        if grad_scale is not None:
            if not (grad_scale.get_device() == p.index and grad_scale.dtype == torch.float32 and grad_scale.numel() == 1):
                raise ValueError("grad_scale must be a float32 CUDA tensor of one element on the parameters' device")
            scale_ptr = grad_scale.data_ptr()
        b1, b2 = self.betas
        rc = capi.load().shampoo_adamw(
            p.ptr, grads.ptr, self._copies_ptr, self._hyper_ptr, p.n, p.segments_ptr, p.nsegments, p.type, grads.type,
            self._state, *self._state_ptrs, self.lr if lr is None else lr, b1, b2, self.eps, self.t + 1, self.seed,
            scale_ptr, _raw_stream(p.index))
        if rc:
            capi.check(rc, "shampoo_adamw")
        self.t += 1

    def moments(self, dtype=torch.float32, stream=None):
        """The values of (m, v) as new flat tensors in the state's layout."""
        p = self.params
        if stream is not None:
            return _on_stream(stream, p.device, lambda: self.moments(dtype), self)
        if p.index != _current_device():
            with torch.cuda.device(p.index):
                return self.moments(dtype)
        if dtype not in _TYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        if self.m_scale is None:
            return self.m.to(dtype, copy=True), self.v.to(dtype, copy=True)
        m, v = torch.empty_like(self.m, dtype=dtype), torch.empty_like(self.v, dtype=dtype)
        mc, vc, ms, vs = self._state_ptrs
        capi.check(capi.shampoo_adamw_moments(mc, ms, vc, vs, m.numel(), m.data_ptr(), v.data_ptr(), _TYPES[dtype],
                                              _raw_stream(p.index)), "shampoo_adamw_moments")
        return m, v

    def state_dict(self):
        """What a resume needs bit for bit: the moments as stored, the layouts of
        the tensors they belong to, the step count and the seed.  Tensors are
        returned as they are."""
        sd = {"m": self.m, "v": self.v, "t": int(self.t), "seed": int(self.seed), "layouts": list(self.params.layouts)}
        if self.m_scale is not None:
            sd.update(m_scale=self.m_scale, v_scale=self.v_scale)
        return sd

    def load_state_dict(self, sd):
        """Restore a state_dict() of an AdamW over tensors of the same layouts, in
        the same order, and the same kind of state.  Saved "layouts" may be
        missing; then only the buffers' sizes are compared.  An error changes
        nothing."""
        names = [k for k in ("m", "v", "m_scale", "v_scale") if getattr(self, k) is not None]
        if {k for k in sd if k not in ("t", "seed", "layouts")} != set(names):
            raise ValueError("the saved moments are of another kind")
        if "layouts" in sd and _nested_tuple(sd["layouts"]) != self.params.layouts:
            raise ValueError("the saved moments are of tensors of other layouts or in another order")
        for name in names:
            dst, src = getattr(self, name), sd[name]
            if tuple(src.shape) != tuple(dst.shape) or src.dtype != dst.dtype:
                raise ValueError(f"{name}: saved {tuple(src.shape)} {src.dtype}, expected "
                                 f"{tuple(dst.shape)} {dst.dtype}")
        t, seed = int(sd["t"]), int(sd["seed"])
        if t < 0 or not 0 <= seed < 1 << 64:
            raise ValueError(f"saved step count {t} or seed {seed} is out of range")
        for name in names:
            getattr(self, name).copy_(sd[name])
        self.t, self.seed = t, seed
