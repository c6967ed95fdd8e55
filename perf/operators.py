"""Timed cases of the AdamW step, the gradient norm and the 4-bit matrix
products: inputs, plain torch forms, float64 values and the work of a pass.

Formats.  Both are microscaled: 32 consecutive elements of a row (or of a
tensor's flat order) share one power-of-two scale 2^(s - 127), held as the
byte s (E8M0; s = 255 stands for NaN).
  MX4   two E2M1 values in a byte, the lower column in the low half; a row is
        padded with zero codes to a multiple of 128 columns.
        s = max(E - 2, 0), E the exponent field of the group's largest
        magnitude (fp32); values round to nearest even and saturate at 6.
  MX8   AdamW's moments, one byte each: m is sign + E4M3 (OCP FP8, bias 7),
        s = max(E - 7, 1); v is unsigned E5M3 (bias 15), s = max(E - 15, 1),
        code 0 becomes 1.  Values round stochastically: with x's place between
        its two neighbours f, the upper one is taken where f + u >= 1,
        u = (h + 1/2) / 65536 and h 16 bits of the element's hash (low half
        for m, high half for v).
A bf16 parameter rounds the same way with the 16 high bits of C2 * hash.  The
hash of an element is a function of (seed, step, position in the state
buffer) alone; every tensor starts at a multiple of 32 there.
"""
import math
import random

import torch

own = False

GROUP = 32
PAD4 = 128
C1, C2, C3, C4 = 0x2F6B4D1D, 0x5A3C91E7, 0x6D41B7A5, 0x3B9F0D4B
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.1
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SHAPES = {"360m": (24, 1024, 4096), "1.3b": (24, 2048, 8192)}  # layers, hidden, MLP


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # The 1-D weights (two norms a layer and the last one) that a block preconditioner leaves to AdamW.
        {"name": "adamw_vectors_f32", "op": "adamw", "shapes": "vectors", "tensors": 49, "largest": 1024,
         "param": "f32", "grad": "f32", "state": "f32", "copy": False, "clip": 0.0},
        # Every weight of the 360M-shaped stack under plain AdamW: fp32 throughout.
        {"name": "adamw_360m_f32", "op": "adamw", "shapes": "360m", "tensors": 0, "largest": 0,
         "param": "f32", "grad": "f32", "state": "f32", "copy": False, "clip": 0.0},
        # Mixed ragged tensors: fp32 masters with a bf16 copy, bf16 gradients, clipped, states in 8 bits.
        {"name": "adamw_mixed_mx8", "op": "adamw", "shapes": "mixed", "tensors": 37, "largest": 4000003,
         "param": "f32", "grad": "bf16", "state": "mx8", "copy": True, "clip": 1.0},
        # The 1.3B-shaped stack without masters: bf16 parameters and gradients, states in 8 bits.
        {"name": "adamw_1p3b_bf16_mx8", "op": "adamw", "shapes": "1.3b", "tensors": 0, "largest": 0,
         "param": "bf16", "grad": "bf16", "state": "mx8", "copy": False, "clip": 0.0},
        # Norm and clip coefficient of a few small gradients, and of the 1.3B-shaped set.
        {"name": "norm_vectors_f32", "op": "norm", "shapes": "vectors", "tensors": 49, "largest": 1024, "grad": "f32"},
        {"name": "norm_1p3b_bf16", "op": "norm", "shapes": "1.3b", "tensors": 0, "largest": 0, "grad": "bf16"},
        # An odd activation matrix grouped along its rows; a weight grouped both ways for training.
        {"name": "quantise_ragged_f32", "op": "quantise", "rows": 333, "cols": 1001, "dtype": "f32", "both": False},
        {"name": "quantise_both_bf16", "op": "quantise", "rows": 16384, "cols": 8192, "dtype": "bf16", "both": True},
        # One token through an MLP-up weight (serving), and an odd product added to an fp32 matrix.
        {"name": "linear_token", "op": "linear", "m": 1, "n": 8192, "k": 2048, "dtype": "bf16"},
        {"name": "product_ragged_f32", "op": "product", "m": 777, "n": 1001, "k": 1537, "out": "f32", "beta": 1.0},
        # 8 sequences of 2048 tokens through MLP-down, already quantised.
        {"name": "product_prompt_bf16", "op": "product", "m": 16384, "n": 2048, "k": 8192, "out": "bf16", "beta": 0.0},
        # Forward and both gradients of the MLP-up layer on 8192 tokens, fp32 master weight.
        {"name": "train_mlp_up", "op": "train", "t": 8192, "n": 8192, "k": 2048, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("adamw", "adamw", "norm", "quantise", "linear", "product", "train"))
    if op in ("adamw", "norm"):
        case = {"op": op, "shapes": "mixed", "tensors": _log(rng, 1, 60), "largest": _log(rng, 100, 12000000),
                "grad": rng.choice(("f32", "bf16"))}
        if op == "adamw":
            case["param"] = rng.choice(("f32", "bf16"))
            case["state"] = rng.choice(("f32", "mx8"))
            case["copy"] = case["param"] == "f32" and rng.random() < 0.5
            case["clip"] = rng.choice((0.0, 1.0))
        return case
    if op == "quantise":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 1, 8192),
                "dtype": rng.choice(("f32", "bf16")), "both": rng.random() < 0.5}
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 2048), "n": _log(rng, 16, 8192), "k": _log(rng, 16, 8192),
                "dtype": rng.choice(("f32", "bf16"))}
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 1, 8192), "k": _log(rng, 1, 8192),
                "out": rng.choice(("f32", "bf16")), "beta": rng.choice((0.0, 1.0))}
    return {"op": op, "t": _log(rng, 16, 8192), "n": _log(rng, 16, 8192), "k": _log(rng, 16, 4096),
            "dtype": rng.choice(("f32", "bf16"))}


def _sizes(case):
    """Element counts of the case's tensors, and which of them are matrices (these decay)."""
    if case["shapes"] in SHAPES:
        layers, h, mlp = SHAPES[case["shapes"]]
        return ([h * h] * 4 + [mlp * h] * 2) * layers, [True] * (6 * layers)
    if case["shapes"] == "vectors":
        return [case["largest"]] * case["tensors"], [False] * case["tensors"]
    r = random.Random(case["tensors"] * 1000003 + case["largest"])
    sizes = [case["largest"]] + [_log(r, 1, case["largest"]) for _ in range(case["tensors"] - 1)]
    return sizes, [r.random() < 0.5 for _ in sizes]


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op in ("adamw", "norm"):
        n = sum(_sizes(case)[0])
        g = size[case["grad"]]
        if op == "norm":
            return {"bytes": g * n + 8, "flops": 2 * n}
        p = size[case["param"]]
        # 8-bit states: codes and scales read and written, and their values written in bf16
        state = 16 if case["state"] == "f32" else 4 + 4 / GROUP + 4
        return {"bytes": (2 * p + g + state + 2 * case["copy"]) * n, "flops": (14 + 2 * (case["clip"] > 0)) * n}
    if op == "quantise":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["dtype"]] + 2 * (1 + case["both"])), "flops": n * (1 + case["both"])}
    per = 0.5 + 1 / GROUP
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": size[case["dtype"]] * (m * k + m * n) + per * n * k, "flops": 2 * m * n * k}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": per * (m + n) * k + size[case["out"]] * m * n * (1 + (case["beta"] != 0)), "flops": 2 * m * n * k}
    t, n, k = case["t"], case["n"], case["k"]
    return {"bytes": 2 * size[case["dtype"]] * (t * k + t * n) + 8 * n * k, "flops": 6 * t * n * k}


# ---------------------------------------------------------------------------
# The formats in 32 bits
# ---------------------------------------------------------------------------

def _wrap(x):
    """The signed 32-bit integer with the low bits of x."""
    return ((x + 0x80000000) & 0xFFFFFFFF) - 0x80000000


def _finish(x):
    """The hash's last steps on 32-bit integers held in int32 tensors (or on one Python integer)."""
    if isinstance(x, int):
        x &= 0xFFFFFFFF
        x = ((x ^ (x >> 16)) * C2) & 0xFFFFFFFF
        x = ((x ^ (x >> 15)) * C3) & 0xFFFFFFFF
        return x ^ (x >> 16)
    x = (x ^ ((x >> 16) & 0xFFFF)) * C2
    x = (x ^ ((x >> 15) & 0x1FFFF)) * C3
    return x ^ ((x >> 16) & 0xFFFF)


def _key(seed, t):
    return _finish(_finish((seed & 0xFFFFFFFF) * C1 + (seed >> 32) * C4) + t * C1)


def _hash(n, seed, t, device, first=0):
    """int32 hashes of positions first ... first + n - 1 of the state buffer."""
    i = torch.arange(first, first + n, device=device, dtype=torch.int64)
    x = ((i & 0xFFFFFFFF) * C1 + (i >> 32) * C4 + _key(seed, t)) & 0xFFFFFFFF
    return _finish(torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32))


def _field(x):
    """Exponent field of the largest magnitude of each group: [groups] int32."""
    return x.abs().view(torch.int32).reshape(-1, GROUP).amax(1) >> 23


def _pow2(field):
    """2^(field - 127) for exponent fields 1 ... 254."""
    return (field << 23).view(torch.float32)


def _encode8(x, rnd16, back, down, signed):
    """Codes (uint8) and scale bytes of x, float32 with a multiple of 32 elements.
    A float32 times 2^-down has the code in its bits 20 ... 27, subnormal codes included."""
    e = _field(x)
    s = torch.clamp(e - back, min=1)
    y = (x.reshape(-1, GROUP) * _pow2(torch.clamp(254 - s, min=1))[:, None]).reshape(-1)
    bits = (y.abs() * 2.0 ** -down).view(torch.int32)
    code = (bits + (rnd16 << 4) + 8) >> 20
    if signed:
        code = code | torch.where(x < 0, 128, 0)
    else:
        code = torch.clamp(code, min=1)
    bad = e == 255
    code = torch.where(bad[:, None], 0, code.reshape(-1, GROUP)).reshape(-1)
    return code.to(torch.uint8), torch.where(bad, 255, s).to(torch.uint8)


def _decode8(code, scale, up, signed):
    c = code.to(torch.int32)
    mag = ((c & (127 if signed else 255)) << 20).view(torch.float32) * 2.0 ** up
    if signed:
        mag = torch.where(c >= 128, -mag, mag)
    s = scale.to(torch.int32)
    f = torch.where(s == 255, float("nan"), _pow2(torch.clamp(s, max=254)))
    return (mag.reshape(-1, GROUP) * f[:, None]).reshape(-1)


def _decode_m(code, scale):
    return _decode8(code, scale, 120, True)


def _decode_v(code, scale):
    return _decode8(code, scale, 112, False)


def _round_bf16(x, rnd16):
    """float32 to bf16, stochastic."""
    bits = (x.view(torch.int32) + rnd16) & -65536
    return torch.where(torch.isnan(x), x, bits.view(torch.float32)).to(torch.bfloat16)


def _values4(x):
    """The MX4 values of each row of x, groups along the row, as float32."""
    x = x.float()
    rows, cols = x.shape
    y = torch.nn.functional.pad(x, (0, -cols % GROUP)).reshape(-1, GROUP)
    e = _field(y)
    s = torch.clamp(e - 2, min=0)
    bad = e == 255
    up = _pow2(torch.clamp(254 - s, min=1))[:, None]
    a = y.abs() * up
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.clamp(torch.round(a / step) * step, max=6.0)
    q = torch.where(y < 0, -a, a) / up
    q = torch.where(bad[:, None], float("nan"), q)
    return q.reshape(rows, -1)[:, :cols]


def _unpack4(codes, scales, cols):
    """float32 [rows, cols] of packed codes [rows, padded / 2] and scale bytes [rows, padded / 32]."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = codes.to(torch.int32)
    v = torch.stack((lut[c & 15], lut[c >> 4]), 2).reshape(codes.shape[0], -1, GROUP)
    s = scales.to(torch.int32)
    f = torch.where(s == 255, float("nan"), torch.where(s == 0, 2.0 ** -127, _pow2(torch.clamp(s, 1, 254))))
    return (v * f[:, :, None]).reshape(codes.shape[0], -1)[:, :cols]


def _pack4(x):
    """Packed codes and scales of x [rows, cols], made when inputs are prepared."""
    rows, cols = x.shape
    q = torch.nn.functional.pad(_values4(x), (0, -cols % PAD4))
    e = _field(torch.nn.functional.pad(x.float(), (0, -cols % PAD4)))
    s = torch.clamp(e - 2, min=0)
    a = (q.reshape(-1, GROUP).abs() * _pow2(254 - s)[:, None]).reshape(rows, -1)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | torch.where(q < 0, 8, 0).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.to(torch.uint8).reshape(rows, -1)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _matrix(gen, rows, cols, std, dtype):
    """Normal values with a spread over the columns and a few large ones, as activations and gradients have."""
    x = torch.randn(rows, cols, generator=gen, device="cuda") * std
    x *= torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 13)
    op = case["op"]
    if own:
        from inverse_root_preconditioning_amd import adamw as AW
        from inverse_root_preconditioning_amd import mx4 as MX
    if op in ("adamw", "norm"):
        sizes, matrix = _sizes(case)
        padded = [-(-n // GROUP) * GROUP for n in sizes]
        first = [sum(padded[:i]) for i in range(len(padded))]
        total = sum(padded)
        real = torch.ones(total, dtype=torch.bool, device="cuda")
        for o, n, m in zip(first, sizes, padded):
            real[o + n:o + m] = False
        std = torch.exp(torch.empty(len(sizes), device="cuda").uniform_(-9, -3, generator=gen))  # a scale for each tensor
        std = torch.repeat_interleave(std, torch.tensor(padded, device="cuda"), output_size=total)
        g = torch.randn(total, generator=gen, device="cuda") * std * real
        st = {"case": case, "seed": seed, "t": 10, "sizes": sizes, "padded": padded, "real": real,
              "grad": g.to(DT[case["grad"]])}
        parts = lambda flat: [flat[o:o + n] for o, n in zip(first, sizes)]  # noqa: E731
        if op == "norm":
            if own:
                st["table"] = AW.TensorTable(parts(st["grad"]))
            return st
        st["param"] = (torch.randn(total, generator=gen, device="cuda") * 0.02 * real).to(DT[case["param"]])
        st["decay"] = [DECAY if m else 0.0 for m in matrix]
        st["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
        m = 0.3 * g + 0.3 * std * torch.randn(total, generator=gen, device="cuda") * real
        v = (std * (0.5 + torch.rand(total, generator=gen, device="cuda"))) ** 2 * real
        del std, g
        if case["state"] == "f32":
            st["m"], st["v"] = m, v
        else:
            h = _hash(total, seed, 0, "cuda")
            st["m"], st["m_scale"] = _encode8(m, h & 0xFFFF, 7, 120, True)
            st["v"], st["v_scale"] = _encode8(v, (h >> 16) & 0xFFFF, 15, 112, False)
            st["v"] *= real
        if own:
            st["opt"] = AW.AdamW(parts(st["param"]), lr=LR, betas=BETAS, eps=EPS, weight_decay=st["decay"],
                                 state=case["state"], copies=parts(st["copy"]) if case["copy"] else None, seed=seed)
            st["opt"].load_state_dict({k: st[k] for k in ("m", "v", "m_scale", "v_scale", "t", "seed") if k in st})
            st["table"] = AW.TensorTable(parts(st["grad"]))
            st["m"] = st["v"] = st["m_scale"] = st["v_scale"] = None
        return st
    if op == "quantise":
        return {"case": case, "x": _matrix(gen, case["rows"], case["cols"], 0.1, DT[case["dtype"]])}
    if op == "train":
        t, n, k, dt = case["t"], case["n"], case["k"], DT[case["dtype"]]
        return {"case": case, "x": _matrix(gen, t, k, 1.0, dt).requires_grad_(own),
                "w": (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).requires_grad_(own),
                "dy": _matrix(gen, t, n, 1e-3, dt)}
    m, n, k = case["m"], case["n"], case["k"]
    w, ws = _pack4(torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k))
    st = {"case": case, "w": w, "w_scale": ws}
    x = _matrix(gen, m, k, 1.0, DT[case.get("dtype", "f32")])
    if own:
        st["wq"] = MX.MX4Matrix(w, ws, n, k)
    if op == "linear":
        st["x"] = x
        return st
    st["a"], st["a_scale"] = _pack4(x)
    st["c"] = torch.randn(m, n, generator=gen, device="cuda").to(DT[case["out"]])
    if own:
        st["aq"] = MX.MX4Matrix(st["a"], st["a_scale"], m, k)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_adamw(s):
    from inverse_root_preconditioning_amd import adamw as AW
    scale = AW.grad_norm(s["table"], s["case"]["clip"])[1:] if s["case"]["clip"] else None
    opt = s["opt"]
    opt.step(s["table"], grad_scale=scale)
    if s["case"]["state"] == "f32":
        m, v = opt.m, opt.v
    else:
        m, v = opt.moments(torch.bfloat16)
    return {"p": s["param"], "copy": s["copy"], "m": m, "v": v}


def _own_norm(s):
    from inverse_root_preconditioning_amd import adamw as AW
    return AW.grad_norm(s["table"], 1.0)


def _own_quantise(s):
    from inverse_root_preconditioning_amd import mx4 as MX
    if s["case"]["both"]:
        q, qt = MX.quantize_both(s["x"])
        return [MX.dequantize(q, torch.bfloat16), MX.dequantize(qt, torch.bfloat16)]
    return [MX.dequantize(MX.quantize(s["x"]), torch.bfloat16)]


def _own_linear(s):
    from inverse_root_preconditioning_amd import mx4 as MX
    return MX.linear(s["x"], s["wq"])


def _own_product(s):
    from inverse_root_preconditioning_amd import mx4 as MX
    return MX.product(s["aq"], s["wq"], out=s["c"], beta=s["case"]["beta"])


def _own_train(s):
    from inverse_root_preconditioning_amd import mx4 as MX
    y = MX.train_linear(s["x"], s["w"])
    dx, dw = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw}


def _norm(g, limit):
    """[norm, factor that brings it down to limit; NaN where the norm is not finite]."""
    norm = (g.float() * g.float()).sum().sqrt()
    c = torch.where(norm > limit, limit / norm, 1.0)
    return torch.stack((norm, torch.where(torch.isfinite(norm), c, float("nan"))))


def _plain_norm(s):
    return _norm(s["grad"], 1.0)


def _plain_adamw(s):
    c = s["case"]
    s["t"] += 1
    t, real, total = s["t"], s["real"], s["real"].numel()
    (b1, b2), n = BETAS, torch.tensor(s["padded"], device="cuda")
    g = s["grad"].float()
    ok = torch.ones((), dtype=torch.bool, device="cuda")
    if c["clip"]:
        scale = _norm(s["grad"], c["clip"])[1]
        g = g * scale
        ok = torch.isfinite(scale)  # a step with a norm that is not finite changes nothing
    low = c["state"] == "mx8"
    m = _decode_m(s["m"], s["m_scale"]) if low else s["m"]
    v = _decode_v(s["v"], s["v_scale"]) if low else s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    del g
    d = m / (v.sqrt() * (1 / math.sqrt(1 - b2 ** t)) + EPS)
    keep = torch.repeat_interleave(1 - LR * torch.tensor(s["decay"], device="cuda"), n, output_size=total)
    p = s["param"].float() * keep - (LR / (1 - b1 ** t)) * d
    del d, keep
    h = _hash(total, s["seed"], t, "cuda") if low or c["param"] == "bf16" else None
    ok = ok & real
    if c["param"] == "bf16":
        p = _round_bf16(p, ((h * C2) >> 16) & 0xFFFF)
    s["param"].copy_(torch.where(ok, p, s["param"]))
    if c["copy"]:
        s["copy"].copy_(torch.where(ok, p.to(torch.bfloat16), s["copy"]))
    del p
    if not low:
        s["m"].copy_(torch.where(ok, m, s["m"]))
        s["v"].copy_(torch.where(ok, v, s["v"]))
        return {"p": s["param"], "copy": s["copy"], "m": s["m"], "v": s["v"]}
    group = ok.reshape(-1, GROUP)[:, 0]
    mc, ms = _encode8(m, h & 0xFFFF, 7, 120, True)
    vc, vs = _encode8(v, (h >> 16) & 0xFFFF, 15, 112, False)
    s["m"].copy_(torch.where(ok, mc, s["m"]))
    s["v"].copy_(torch.where(ok, vc, s["v"]))
    s["m_scale"].copy_(torch.where(group, ms, s["m_scale"]))
    s["v_scale"].copy_(torch.where(group, vs, s["v_scale"]))
    return {"p": s["param"], "copy": s["copy"], "m": _decode_m(s["m"], s["m_scale"]).to(torch.bfloat16),
            "v": _decode_v(s["v"], s["v_scale"]).to(torch.bfloat16)}


def _plain_quantise(s):
    x = s["x"]
    q = [_values4(x).to(torch.bfloat16)]
    if s["case"]["both"]:
        q.append(_values4(x.t().contiguous()).to(torch.bfloat16))
    return q


def _plain_linear(s):
    w = _unpack4(s["w"], s["w_scale"], s["case"]["k"])
    return (_values4(s["x"]) @ w.t()).to(s["x"].dtype)


def _plain_product(s):
    k = s["case"]["k"]
    c = _unpack4(s["a"], s["a_scale"], k) @ _unpack4(s["w"], s["w_scale"], k).t()
    if s["case"]["beta"]:
        c = c + s["case"]["beta"] * s["c"].float()
    s["c"].copy_(c)
    return s["c"]


def _plain_train(s):
    x, w, dy = s["x"], s["w"], s["dy"]
    y = _values4(x) @ _values4(w).t()
    dx = _values4(dy) @ _values4(w.t().contiguous()).t()
    dw = _values4(dy.t().contiguous()) @ _values4(x.t().contiguous()).t()
    return {"y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw}


_OWN = {"adamw": _own_adamw, "norm": _own_norm, "quantise": _own_quantise, "linear": _own_linear,
        "product": _own_product, "train": _own_train}
_PLAIN = {"adamw": _plain_adamw, "norm": _plain_norm, "quantise": _plain_quantise, "linear": _plain_linear,
          "product": _plain_product, "train": _plain_train}


# ---------------------------------------------------------------------------
# The same in 64 bits
# ---------------------------------------------------------------------------

def _times2(x, e):
    """x 2^e for float64 x, the power made from its bits."""
    return x * ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values4(x):
    """Nearest multiple of the spacing that holds at each magnitude: E2M1 has one mantissa bit from 1 up to 6."""
    x = x.double()
    rows, cols = x.shape
    y = torch.nn.functional.pad(x, (0, -cols % GROUP)).reshape(rows, -1, GROUP)
    top = torch.frexp(y.abs().amax(2, keepdim=True))[1] - 1  # floor(log2) of the largest
    s = torch.clamp(top - 2, min=-127)
    a = _times2(y, -s)
    e = torch.clamp(torch.frexp(a)[1] - 1, 0, 2)
    q = _times2(torch.round(_times2(a, 1 - e)), e - 1).clamp(-6, 6)
    return _times2(q, s).reshape(rows, -1)[:, :cols]


def _exact_codes8(x, h16, top_at, lowest, floor):
    """x rounded to 3 mantissa bits below its exponent, which is at least `lowest` where the group's largest has `top_at`."""
    y = x.reshape(-1, GROUP)
    big = torch.frexp(y.abs().amax(1, keepdim=True))[1] - 1
    s = torch.clamp(big - top_at, min=-126)
    a = _times2(y.abs(), -s)
    step = _times2(torch.ones_like(a), torch.clamp(torch.frexp(a)[1] - 1, min=lowest) - 3)
    q = torch.floor(a / step + (h16.double().reshape(-1, GROUP) + 0.5) / 65536) * step
    if floor:
        q = torch.clamp(q, min=2.0 ** (lowest - 3))
    return _times2(torch.where(y < 0, -q, q), s).reshape(-1)


def _exact_state8(code, scale, bias, signed):
    """Values of stored codes: exponent field, three mantissa bits, the group's power of two."""
    c = code.long()
    mag = c & 127 if signed else c
    e, f = mag >> 3, (mag & 7).double() / 8
    v = _times2(torch.where(e > 0, 1 + f, f), torch.clamp(e, min=1) - bias)
    v = torch.where(c >= 128, -v, v) if signed else v
    return _times2(v.reshape(-1, GROUP), scale.long()[:, None] - 127).reshape(-1)


def _exact_adamw(case, seed):
    global own
    was, own = own, False  # inputs and states as plain tensors
    try:
        s = prepare(case, seed)
    finally:
        own = was
    (b1, b2), t, total = BETAS, s["t"] + 1, s["real"].numel()
    low = case["state"] == "mx8"
    c = 1.0
    if case["clip"]:
        c = min(1.0, case["clip"] / math.sqrt(sum(float((x.double() ** 2).sum()) for x in s["grad"].split(1 << 26))))
    decay = torch.repeat_interleave(torch.tensor(s["decay"], dtype=torch.float64, device="cuda"),
                                    torch.tensor(s["padded"], device="cuda"), output_size=total)
    p_out, m_out, v_out = (torch.empty(total, dtype=torch.float64, device="cuda") for _ in range(3))
    for a in range(0, total, 1 << 26):
        z = min(total, a + (1 << 26))
        part, ga, gz = slice(a, z), a // GROUP, z // GROUP
        g, real = s["grad"][part].double() * c, s["real"][part]
        if low:
            m = _exact_state8(s["m"][part], s["m_scale"][ga:gz], 7, True)
            v = _exact_state8(s["v"][part], s["v_scale"][ga:gz], 15, False)
        else:
            m, v = s["m"][part].double(), s["v"][part].double()
        m1 = b1 * m + (1 - b1) * g
        v1 = b2 * v + (1 - b2) * g * g
        p = s["param"][part].double()
        d = (m1 / (1 - b1 ** t)) / (torch.sqrt(v1 / (1 - b2 ** t)) + EPS)
        p_out[part] = torch.where(real, p - LR * (decay[part] * p + d), p)
        if low:
            h = _hash(z - a, seed, t, "cuda", a)
            m1 = _exact_codes8(m1, h & 0xFFFF, 7, -6, False)
            v1 = _exact_codes8(v1, (h >> 16) & 0xFFFF, 15, -14, True)
        m_out[part] = torch.where(real, m1, m)
        v_out[part] = torch.where(real, v1, v)
    return {"p": p_out, "copy": p_out if case["copy"] else None, "m": m_out, "v": v_out}


def exact(case, seed):
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(case, seed)
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if op == "norm":
        norm = math.sqrt(sum(float((x.double() ** 2).sum()) for x in s["grad"].split(1 << 26)))
        return torch.tensor([norm, min(1.0, 1.0 / norm)], dtype=torch.float64)
    if op == "quantise":
        q = [_exact_values4(s["x"])]
        return q + [_exact_values4(s["x"].t())] if case["both"] else q
    if op == "train":
        x, w, dy = s["x"], s["w"], s["dy"]
        return {"y": _exact_values4(x) @ _exact_values4(w).t(),
                "dx": _exact_values4(dy) @ _exact_values4(w.t()).t(),
                "dw": _exact_values4(dy.t()) @ _exact_values4(x.t()).t()}
    k = case["k"]
    w = _unpack4(s["w"], s["w_scale"], k).double()  # exact in either width
    if op == "linear":
        return _exact_values4(s["x"]) @ w.t()
    c = _unpack4(s["a"], s["a_scale"], k).double() @ w.t()
    return c + case["beta"] * s["c"].double()
