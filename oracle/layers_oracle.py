"""Float64 oracle of the MX8 rows, activations, norms and joins (torch on the
CPU), written from their definitions.  Test infrastructure only.

`magnitude=True` evaluates the same formulas with every term's absolute value
added: n fp32 operations leave an error of at most about n 2^-24 of that."""
import math
from types import SimpleNamespace

import torch

GROUP = 32
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "relu2")


def mx8_codes(x):
    """(codes, scales) of the rows of x [rows, cols] as int64, padded to 32 columns."""
    rows, cols = x.shape
    y = torch.nn.functional.pad(x.double(), (0, -cols % GROUP)).reshape(rows, -1, GROUP)
    top = y.abs().amax(2)
    bad = ~torch.isfinite(y).all(2)
    # the exponent field as fp32 has it: 0 for subnormals, which are below 2^-126
    field = torch.where(top >= 2.0 ** -126, torch.frexp(torch.where(bad, 1.0, top))[1].long() + 126, 0)
    s = torch.where(bad, 255, torch.clamp(field - 7, min=1))
    a = torch.ldexp(torch.where(bad[..., None], 0.0, y.abs()), (127 - torch.where(bad, 127, s))[..., None])
    e = torch.clamp(torch.frexp(a)[1] - 1, min=-6)
    m = torch.round(torch.ldexp(a, 3 - e)).long()          # 0 ... 16, to nearest even
    e, m = torch.where(m == 16, e + 1, e), torch.where(m == 16, 8, m)
    code = torch.where(m >= 8, (e.long() + 7) * 8 + m - 8, m)
    code = code + 128 * (torch.copysign(torch.ones_like(y), y) < 0)
    code = torch.where(bad[..., None], 0x7f, code)
    return code.reshape(rows, -1), s


def mx8_decode(codes, scales, cols):
    c = codes.long().reshape(codes.shape[0], -1, GROUP)
    e, m = (c & 127) >> 3, (c & 7).double()
    v = torch.where(e > 0, torch.ldexp(8 + m, e - 10), torch.ldexp(m, torch.tensor(-9)))
    v = torch.where(c >= 128, -v, v)
    s = scales.long()[..., None]
    v = torch.where(s == 255, math.nan, torch.ldexp(v, s - 127))
    return v.reshape(codes.shape[0], -1)[:, :cols]


def mx8_values(x):
    flat = x.reshape(-1, x.shape[-1])
    return mx8_decode(*mx8_codes(flat), flat.shape[1]).reshape(x.shape)


def kept(x, keep):
    return mx8_values(x) if keep == "mx8" else x.double()


def act(x, name):
    """(f(x), f'(x))"""
    x = x.double()
    if name == "relu":
        return x.clamp(min=0), (x > 0).double()
    if name == "relu2":
        return x.clamp(min=0) ** 2, 2 * x.clamp(min=0)
    if name == "gelu":
        p, d = torch.erfc(-x * math.sqrt(0.5)) / 2, torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    else:
        v, dv = x, 1.0
        if name == "gelu_tanh":
            v, dv = math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3), math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * x ** 2)
        p = torch.sigmoid(v)
        d = p * torch.sigmoid(-v) * dv
    return x * p, p + x * d


def _row_mean(x, magnitude=False):
    return (x.abs() if magnitude else x).mean(-1, keepdim=True)


def stats(x, kind, eps):
    """mean (0 for RMS) and s of each row"""
    mean = _row_mean(x) if kind == "layer" else torch.zeros_like(x[..., :1])
    return mean, 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)


def _sub(a, b, magnitude):
    return a.abs() + b.abs() if magnitude else a - b


def join(r, y, n1=None, gate=None, scale=1.0, n2=None, magnitude=False):
    """h, u and the statistics; n1, n2: (kind, weight, bias, eps), weight and bias may be None."""
    o = SimpleNamespace(st1=None, st2=None, u=None)
    ab = (lambda t: t.abs()) if magnitude else (lambda t: t)  # noqa: E731

    def normed(x, xm, n):
        mean, s = stats(x, n[0], n[3])
        # x - mean carries the error of the mean, which is that of a sum of magnitudes
        v = (xm.abs() + _row_mean(xm, True) if n[0] == "layer" else xm.abs()) * s if magnitude else (x - mean) * s
        if n[1] is not None:
            v = v * ab(n[1].double())
        if n[2] is not None:
            v = v + ab(n[2].double())
        return v, (mean, s)

    r = r.double()
    if y is None:
        o.h, hm = r, ab(r)
    else:
        y = y.double()
        z, zt = ab(y), y
        if n1 is not None:
            z, o.st1 = normed(y, y, n1)
            zt = join(y, None, n2=n1).u if magnitude else z
        g = 1.0 if gate is None else gate.double()
        o.h = hm = abs(scale) * ab(r) + (ab(g) if gate is not None else 1.0) * z if magnitude else scale * r + g * z
        true = scale * r + g * zt
        if magnitude:
            o.true_h = true
    if n2 is not None:
        base = (o.h if y is None else o.true_h) if magnitude else o.h
        o.u, o.st2 = normed(base, hm, n2)
    return o


def join_backward(r, y, st1, st2, n1=None, gate=None, scale=1.0, n2=None, dh=None, du=None, magnitude=False):
    """Gradients by name at the inputs r, y with the given statistics."""
    g = SimpleNamespace(r=None, y=None, w1=None, b1=None, gate=None, w2=None, b2=None)
    ab = (lambda t: t.abs()) if magnitude else (lambda t: t)  # noqa: E731
    cols = r.shape[-1]
    rows = lambda t: t.reshape(-1, cols).sum(0)  # noqa: E731

    def normed(x, st, n):
        mean, s = st
        return (_sub(x, mean, magnitude) + (_row_mean(x, True) if magnitude and n[0] == "layer" else 0)) * s

    def back(grad, xn, st, n):
        w = 1.0 if n[1] is None else ab(n[1].double())
        q = grad * w
        along = xn * _row_mean(q * xn)
        d = q + along if magnitude else q - along
        if n[0] == "layer":
            d = d + _row_mean(q) if magnitude else d - _row_mean(q)
        return d * st[1]

    r = ab(r.double())
    total = torch.zeros_like(r) if dh is None else ab(dh.double())
    yn = z = None
    gt = 1.0 if gate is None else ab(gate.double())
    if y is not None:
        yn = z = ab(y.double())
        if n1 is not None:
            yn = z = normed(y.double(), st1, n1)
            if n1[1] is not None:
                z = z * ab(n1[1].double())
            if n1[2] is not None:
                z = z + ab(n1[2].double())
    if du is not None:
        du = ab(du.double())
        h = r if y is None else abs(scale) * r + gt * z if magnitude else scale * r + gt * z
        hn = normed(h, st2, n2)
        total = total + back(du, hn, st2, n2)
        g.w2, g.b2 = rows(du * hn), rows(du)
    if y is None:
        g.r = total
        return g
    g.r = (abs(scale) if magnitude else scale) * total
    dz = gt * total
    g.y = dz
    if n1 is not None:
        g.y = back(dz, yn, st1, n1)
        g.w1, g.b1 = rows(dz * yn), rows(dz)
    if gate is not None:
        full = total * z
        g.gate = full.sum_to_size(gate.shape) if gate.dim() == full.dim() else rows(full)
    return g
