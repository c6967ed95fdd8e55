"""Float64 oracle of the AdamW step, the gradient norm and the MX4 matrices.

Written from the formulas in numpy, apart from the package; test
infrastructure only.  Numbers are exact in float64 up to its own rounding, so
every rounding to fewer bits below is the one the format defines.
"""
import math

import numpy as np

GROUP = 32
MASK = 0xFFFFFFFF


# ---------------------------------------------------------------------------
# The hash of a state position
# ---------------------------------------------------------------------------

def _finish(x):
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x5A3C91E7)) & np.uint64(MASK)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x6D41B7A5)) & np.uint64(MASK)
    return x ^ (x >> np.uint64(16))


def position_hash(pos, seed, step):
    """32-bit hashes (uint64 array) of state positions for one step of one seed."""
    with np.errstate(over="ignore"):
        key = _finish(np.uint64(((seed & MASK) * 0x2F6B4D1D + (seed >> 32) * 0x3B9F0D4B) & MASK))
        key = _finish(np.uint64((int(key) + step * 0x2F6B4D1D) & MASK))
        pos = np.asarray(pos, dtype=np.uint64)
        x = (pos & np.uint64(MASK)) * np.uint64(0x2F6B4D1D) + (pos >> np.uint64(32)) * np.uint64(0x3B9F0D4B) + key
        return _finish(x & np.uint64(MASK))


# ---------------------------------------------------------------------------
# 8-bit moments
# ---------------------------------------------------------------------------

M8 = dict(back=7, bias=7, signed=True)
V8 = dict(back=15, bias=15, signed=False)


def _floor_log2(a):
    return np.frexp(a)[1] - 1


def mx8_encode(x, h16, back, bias, signed):
    """(codes, scale bytes) of x (float64, a multiple of 32 elements) with 16-bit hashes h16."""
    y = np.asarray(x, dtype=np.float64).reshape(-1, GROUP)
    h = np.asarray(h16, dtype=np.float64).reshape(-1, GROUP)
    bad = ~np.isfinite(y).all(axis=1)
    y = np.where(bad[:, None], 0.0, y)
    top = np.abs(y).max(axis=1)
    field = np.where(top > 0, np.clip(_floor_log2(np.where(top > 0, top, 1.0)) + 127, 0, 254), 0)
    s = np.maximum(field - back, 1)
    a = np.ldexp(np.abs(y), 127 - s[:, None])
    e = np.maximum(_floor_log2(np.where(a > 0, a, 1e-300)), 1 - bias)
    n = np.floor(np.ldexp(a, 3 - e) + (h + 0.5) / 65536)       # in eighths of 2^e
    code = np.where(n >= 16, (e + 1 + bias) * 8, np.where(n >= 8, (e + bias) * 8 + (n - 8), n)).astype(np.int64)
    code = code | np.where(y < 0, 128, 0) if signed else np.maximum(code, 1)
    code = np.where(bad[:, None], 0, code)
    return code.reshape(-1).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def mx8_decode(code, scale, back, bias, signed):
    c = np.asarray(code, dtype=np.int64).reshape(-1, GROUP)
    mag = c & 127 if signed else c
    e, f = mag >> 3, mag & 7
    v = np.where(e > 0, np.ldexp(8.0 + f, np.maximum(e, 1) - bias - 3), np.ldexp(f * 1.0, 1 - bias - 3))
    v = np.where(c >= 128, -v, v) if signed else v
    s = np.asarray(scale, dtype=np.int64)
    v = np.ldexp(v, s[:, None] - 127)
    return np.where((s == 255)[:, None], np.nan, v).reshape(-1)


# ---------------------------------------------------------------------------
# AdamW and the norm
# ---------------------------------------------------------------------------

def adamw(p, g, m, v, lr, b1, b2, eps, decay, step, coef=1.0):
    """One step in float64: (p, m, v)."""
    p, g, m, v = (np.asarray(t, dtype=np.float64) for t in (p, g, m, v))
    g = g * coef
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    d = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p - lr * decay * p - lr * d, m, v


def round_bf16(x, h16):
    """x as bf16 values, stochastically: of two neighbours the one farther from 0 where f + (h + 1/2) / 65536 >= 1."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    e = np.maximum(_floor_log2(np.where(a > 0, a, 1e-300)), -126) - 7       # of the spacing
    n = np.floor(np.ldexp(a, -e) + (np.asarray(h16, dtype=np.float64) + 0.5) / 65536)
    return np.copysign(np.ldexp(n, e), x)


def grad_norm(tensors, max_norm):
    """(norm, clipping factor)."""
    n = math.sqrt(sum(float((np.asarray(t, dtype=np.float64) ** 2).sum()) for t in tensors))
    return n, min(1.0, max_norm / n) if n > 0 else 1.0


# ---------------------------------------------------------------------------
# MX4
# ---------------------------------------------------------------------------

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize(x):
    """(4-bit codes [rows, 32 ceil(cols / 32)], scale bytes) of x, groups along its rows."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    y = np.pad(x, ((0, 0), (0, -cols % GROUP))).reshape(rows, -1, GROUP)
    bad = ~np.isfinite(y).all(axis=2)
    y = np.where(bad[..., None], 0.0, y)
    top = np.abs(y).max(axis=2)
    # the exponent field of a float32: 0 for zero and its subnormals
    field = np.where(top > 0, np.maximum(_floor_log2(np.where(top > 0, top, 1.0)) + 127, 0), 0)
    s = np.maximum(field - 2, 0)
    a = np.ldexp(np.abs(y), 127 - s[..., None])
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.zeros(a.shape, dtype=np.int64)
    for i, t in enumerate(mid):   # value i + 1 from the midpoint on; on it only if i + 1 is even
        code = np.where((a > t) | ((a == t) & ((i + 1) % 2 == 0)), i + 1, code)
    code = np.where(y < 0, code + 8, code)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(rows, -1).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def mx4_values(code, scale, cols):
    c = np.asarray(code, dtype=np.int64)
    rows = c.shape[0]
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.asarray(scale, dtype=np.int64)
    v = np.ldexp(v.reshape(rows, -1, GROUP), s[..., None] - 127)
    v = np.where((s == 255)[..., None], np.nan, v)
    return v.reshape(rows, -1)[:, :cols]


def mx4_round(x):
    """The values that x is quantised to."""
    code, s = mx4_quantize(x)
    return mx4_values(code, s, np.asarray(x).shape[1])
