"""Timed cases of the layers between the linear ones: 8-bit activation
checkpoints, activations and gated activations, norms, and the joins of a block
with its residual; inputs, plain torch forms, float64 values and the work of a
pass.

MX8 rows: 32 consecutive columns share a power of two 2^(s - 127), held as the
byte s; values are sign + E4M3 (OCP FP8), rounded to nearest even after division
by it.  s = max(E - 7, 1), E the exponent field of the group's largest
magnitude (fp32), so that nothing saturates; s = 255 stands for a group with an
entry that is not finite, whose values are all NaN.

Where "keep" is "mx8", the backward pass takes the inputs (an activation's, a
norm's, a join's residual and branch) from their MX8 values and forms from them
what else it needs; the outputs and the row statistics are those of the inputs
as they are.
"""
import math

import torch

own = False

GROUP = 32
EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "relu2")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # An odd activation matrix to 8 bits and back; the MLP activations of 8 sequences of 2048 tokens.
        {"name": "mx8_ragged_f32", "op": "mx8", "rows": 777, "cols": 1001, "dtype": "f32"},
        {"name": "mx8_mlp_bf16", "op": "mx8", "rows": 16384, "cols": 8192, "dtype": "bf16"},
        # The MLP's activation for one token (serving).
        {"name": "act_token", "op": "act", "rows": 1, "cols": 8192, "act": "gelu", "gated": False, "train": False,
         "keep": "same", "dtype": "bf16"},
        # An odd MLP in fp32, forward and backward.
        {"name": "act_ragged_f32", "op": "act", "rows": 1001, "cols": 1537, "act": "gelu", "gated": False,
         "train": True, "keep": "same", "dtype": "f32"},
        # Gated MLP of 4 sequences of 2048 tokens, both halves from one product, inputs kept in 8 bits.
        {"name": "gated_train_mx8", "op": "act", "rows": 8192, "cols": 8192, "act": "silu", "gated": True,
         "train": True, "keep": "mx8", "dtype": "bf16"},
        # The norm before a block: one token; an odd LayerNorm; 8 sequences of 2048 tokens, kept in 8 bits.
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 2048, "kind": "rms", "bias": False, "train": False,
         "keep": "same", "stream": "bf16", "branch": "bf16", "param": "f32"},
        {"name": "norm_ragged_f32", "op": "norm", "rows": 333, "cols": 1001, "kind": "layer", "bias": True,
         "train": True, "keep": "same", "stream": "f32", "branch": "f32", "param": "f32"},
        {"name": "norm_train_mx8", "op": "norm", "rows": 16384, "cols": 2048, "kind": "rms", "bias": False,
         "train": True, "keep": "mx8", "stream": "bf16", "branch": "bf16", "param": "f32"},
        # A block's output joined to the residual stream and normed for the next block: one token; an fp32 stream
        # with bf16 branches over a prompt; odd sequences with a gate each; training with 8-bit checkpoints.
        {"name": "join_token", "op": "join", "seqs": 1, "len": 1, "cols": 2048, "after": "rms", "before": "rms",
         "bias": False, "gate": "channel", "train": False, "keep": "same", "stream": "bf16", "branch": "bf16",
         "param": "f32"},
        {"name": "join_prompt_mixed", "op": "join", "seqs": 8, "len": 2048, "cols": 2048, "after": "none",
         "before": "rms", "bias": False, "gate": "none", "train": False, "keep": "same", "stream": "f32",
         "branch": "bf16", "param": "f32"},
        {"name": "join_ragged_f32", "op": "join", "seqs": 7, "len": 143, "cols": 1537, "after": "layer",
         "before": "layer", "bias": True, "gate": "sequence", "train": True, "keep": "same", "stream": "f32",
         "branch": "f32", "param": "f32"},
        {"name": "join_train_mx8", "op": "join", "seqs": 8, "len": 2048, "cols": 2048, "after": "rms",
         "before": "rms", "bias": False, "gate": "channel", "train": True, "keep": "mx8", "stream": "bf16",
         "branch": "bf16", "param": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("mx8", "act", "act", "norm", "norm", "join", "join", "join"))
    cols = _log(rng, 16, 8192)
    rows = _log(rng, 1, min(16384, (1 << 24) // cols))
    if op == "mx8":
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(("f32", "bf16"))}
    train = rng.random() < 0.7
    case = {"op": op, "cols": cols, "train": train, "keep": rng.choice(("same", "mx8")) if train else "same"}
    if op == "act":
        return {**case, "rows": rows, "act": rng.choice(ACTS), "gated": rng.random() < 0.5,
                "dtype": rng.choice(("f32", "bf16"))}
    stream, branch = rng.choice((("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")))
    case = {**case, "stream": stream, "branch": branch, "param": rng.choice(("f32", "bf16")),
            "bias": rng.random() < 0.3}
    if op == "norm":
        return {**case, "rows": rows, "kind": rng.choice(("rms", "rms", "layer"))}
    seqs = _log(rng, 1, min(rows, 16))
    return {**case, "seqs": seqs, "len": rows // seqs, "after": rng.choice(("none", "rms", "layer")),
            "before": rng.choice(("none", "rms", "rms", "layer")),
            "gate": rng.choice(("none", "channel", "sequence", "token"))}


def work(case):
    op, cols = case["op"], case["cols"]
    n = case.get("rows", case.get("seqs", 0) * case.get("len", 0)) * cols
    if op == "mx8":  # one way and the other: codes are written and read
        return {"bytes": n * 2 * (SIZE[case["dtype"]] + 1 + 1 / GROUP), "flops": 4 * n}
    if op == "act":
        inputs = 1 + case["gated"]
        # forward: inputs and y; backward besides: dy and the inputs' gradients
        return {"bytes": n * SIZE[case["dtype"]] * (inputs + 1) * (1 + case["train"]),
                "flops": n * (10 + 15 * case["train"])}
    s, b = SIZE[case["stream"]], SIZE[case["branch"]]
    if op == "norm":
        return {"bytes": n * (s + b) * (1 + case["train"]), "flops": n * (6 + 12 * case["train"])}
    each = 2 * s + b * (2 if case["before"] != "none" else 1)
    return {"bytes": n * each * (1 + case["train"]), "flops": n * (14 + 30 * case["train"])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, cols, std, dtype):
    """Normal values with a spread over the columns and a few large ones, as activations and gradients have."""
    x = _normal(gen, rows, cols) * std
    x *= torch.exp(0.5 * _normal(gen, cols))
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    op, cols = case["op"], case["cols"]
    train = case.get("train", False)
    leaf = (lambda t: t.requires_grad_(own and train))  # noqa: E731
    if op == "mx8":
        return {"case": case, "x": _activations(gen, case["rows"], cols, 1.0, DT[case["dtype"]])}
    if op == "act":
        rows, dt = case["rows"], DT[case["dtype"]]
        return {"case": case, "x": leaf(_activations(gen, rows, cols * (1 + case["gated"]), 1.0, dt)),
                "dy": _activations(gen, rows, cols, 1e-3, dt) if train else None}
    stream, branch, param = DT[case["stream"]], DT[case["branch"]], DT[case["param"]]
    st = {"case": case}

    def parameters(kind, tag):
        if kind != "none":
            st["w" + tag] = leaf((1 + 0.1 * _normal(gen, cols)).to(param))
            if case["bias"]:
                st["b" + tag] = leaf((0.1 * _normal(gen, cols)).to(param))

    if op == "norm":
        st["x"] = leaf(_activations(gen, case["rows"], cols, 2.0, stream))
        parameters(case["kind"], "2")
        st["du"] = _activations(gen, case["rows"], cols, 1e-3, branch) if train else None
    else:
        seqs, n = case["seqs"], case["len"]
        shape = (seqs, n, cols)
        st["r"] = leaf(_activations(gen, seqs * n, cols, 2.0, stream).view(shape))
        st["y"] = leaf(_activations(gen, seqs * n, cols, 0.5, branch).view(shape))
        parameters(case["after"], "1")
        parameters(case["before"], "2")
        if case["gate"] != "none":
            size = {"channel": (cols,), "sequence": (seqs, 1, cols), "token": (seqs, n, 1)}[case["gate"]]
            st["g"] = leaf((0.5 + 0.25 * _normal(gen, *size)).to(param))
        st["scale"] = 0.875
        if train:
            st["dh"] = _activations(gen, seqs * n, cols, 1e-3, stream).view(shape)
            if case["before"] != "none":
                st["du"] = _activations(gen, seqs * n, cols, 1e-3, branch).view(shape)
    if own:
        from inverse_root_preconditioning_amd import layers as L

        def norm(kind, tag):
            return L.Norm(kind, st.get("w" + tag), st.get("b" + tag), EPS) if kind != "none" else None
        st["norm1"] = norm(case.get("after", "none"), "1")
        st["norm2"] = norm(case["kind"] if op == "norm" else case["before"], "2")
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

PARAMETERS = ("w1", "b1", "g", "w2", "b2")


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_mx8(s):
    from inverse_root_preconditioning_amd import mx8 as M8
    return M8.dequantize(M8.quantize(s["x"]), s["x"].dtype)


def _own_act(s):
    from inverse_root_preconditioning_amd import layers as L
    c = s["case"]
    y = (L.gated if c["gated"] else L.activation)(s["x"], act=c["act"], keep=c["keep"])
    if not c["train"]:
        return {"y": y}
    return {"y": y.detach(), "dx": torch.autograd.grad(y, s["x"], s["dy"])[0]}


def _own_norm(s):
    from inverse_root_preconditioning_amd import layers as L
    c = s["case"]
    u = L.norm(s["x"], s["norm2"], dtype=DT[c["branch"]], keep=c["keep"])
    if not c["train"]:
        return {"u": u}
    names = ["x"] + [p for p in PARAMETERS if p in s]
    return {"u": u.detach(), **dict(zip(names, torch.autograd.grad(u, [s[n] for n in names], s["du"])))}


def _own_join(s):
    from inverse_root_preconditioning_amd import layers as L
    c = s["case"]
    h, u = L.join(s["r"], s["y"], after=s["norm1"], gate=s.get("g"), scale=s["scale"], before=s["norm2"],
                  keep=c["keep"])
    if not c["train"]:
        return {"h": h, "u": u}
    names = ["r", "y"] + [p for p in PARAMETERS if p in s]
    outs, grads = ((h,), (s["dh"],)) if u is None else ((h, u), (s["dh"], s["du"]))
    return {"h": h.detach(), "u": None if u is None else u.detach(),
            **dict(zip(names, torch.autograd.grad(outs, [s[n] for n in names], grads)))}


def _pow2(field):
    """2^(field - 127) for exponent fields 1 ... 254."""
    return (field << 23).view(torch.float32)


def _values8(x):
    """The MX8 values of each row of x, as float32."""
    x = x.float()
    cols = x.shape[-1]
    y = torch.nn.functional.pad(x.reshape(-1, cols), (0, -cols % GROUP)).reshape(-1, GROUP)
    e = y.abs().view(torch.int32).amax(1) >> 23
    s = torch.clamp(e - 7, min=1)
    bad = e == 255
    a = y.abs() * _pow2(torch.clamp(254 - s, min=1))[:, None]
    step = _pow2(torch.clamp(a.view(torch.int32) >> 23, 121, 150) - 3)  # normal from 2^-6 on
    q = torch.round(a / step) * step * _pow2(torch.clamp(s, max=254))[:, None]
    q = torch.where(y < 0, -q, q)
    q = torch.where(bad[:, None], float("nan"), q)
    return q.reshape(-1, cols + -cols % GROUP)[:, :cols].reshape(x.shape)


def _kept(x, case):
    return _values8(x) if case["keep"] == "mx8" else x.float()


def _plain_mx8(s):
    return _values8(s["x"]).to(s["x"].dtype)


SQRT_HALF, RSQRT_2PI = math.sqrt(0.5), 1 / math.sqrt(2 * math.pi)
TANH_A, TANH_B = math.sqrt(2 / math.pi), 0.044715


def _act(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * 0.5 * torch.erfc(-x * SQRT_HALF)
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * TANH_A * (x + TANH_B * x * x * x))
    r = torch.clamp(x, min=0)
    return r if act == "relu" else r * r


def _act_slope(x, act):
    if act == "silu":
        p = torch.sigmoid(x)
        return p * (1 + x * (1 - p))
    if act == "gelu":
        return 0.5 * torch.erfc(-x * SQRT_HALF) + x * torch.exp(-0.5 * x * x) * RSQRT_2PI
    if act == "gelu_tanh":
        p = torch.sigmoid(2 * TANH_A * (x + TANH_B * x * x * x))
        return p + x * p * (1 - p) * (2 * TANH_A) * (1 + 3 * TANH_B * x * x)
    return (x > 0).to(x.dtype) if act == "relu" else 2 * torch.clamp(x, min=0)


def _plain_act(s):
    c, x, dt = s["case"], s["x"], s["x"].dtype
    f = c["cols"]
    a = x[:, :f].float()
    y = _act(a, c["act"])
    if c["gated"]:
        y = y * x[:, f:].float()
    y = y.to(dt)
    if not c["train"]:
        return {"y": y}
    a, dy = _kept(x[:, :f], c), s["dy"].float()
    if not c["gated"]:
        return {"y": y, "dx": (dy * _act_slope(a, c["act"])).to(dt)}
    b = _kept(x[:, f:], c)
    return {"y": y, "dx": torch.cat((dy * b * _act_slope(a, c["act"]), dy * _act(a, c["act"])), 1).to(dt)}


def _norm(x, kind, w, b):
    """Output, mean (0 for RMS) and 1 / root of each row."""
    mu = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    d = x - mu
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    u = d * r * w.float()
    return (u if b is None else u + b.float()), mu, r


def _norm_back(du, x, mu, r, kind, w):
    """Gradient of the input; normed input."""
    xn = (x - mu) * r
    g = du * w.float()
    dx = g - xn * (g * xn).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(-1, keepdim=True)
    return dx * r, xn


def _rows(t):
    return t.reshape(-1, t.shape[-1]).sum(0)


def _plain_norm(s):
    c, x = s["case"], s["x"]
    w, b, kind = s.get("w2"), s.get("b2"), c["kind"]
    u, mu, r = _norm(x.float(), kind, w, b)
    u = u.to(DT[c["branch"]])
    if not c["train"]:
        return {"u": u}
    du = s["du"].float()
    dx, xn = _norm_back(du, _kept(x, c), mu, r, kind, w)
    out = {"u": u, "x": dx.to(x.dtype), "w2": _rows(du * xn).to(w.dtype)}
    if b is not None:
        out["b2"] = _rows(du).to(w.dtype)
    return out


def _join_forward(s, r, y):
    """h, u, the gate and the statistics of both norms."""
    c = s["case"]
    z, mu1, r1 = (y, None, None) if c["after"] == "none" else _norm(y, c["after"], s.get("w1"), s.get("b1"))
    g = s["g"].float() if "g" in s else None
    h = s["scale"] * r + (z if g is None else g * z)
    u, mu2, r2 = (None, None, None) if c["before"] == "none" else _norm(h, c["before"], s.get("w2"), s.get("b2"))
    return h, u, g, (mu1, r1), (mu2, r2)


def _join_back(s, dh, du, r, y, g, n1, n2):
    """Gradients by name, from kept r and y."""
    c, out = s["case"], {}
    z = y
    if c["after"] != "none":
        yn = (y - n1[0]) * n1[1]
        z = yn * s["w1"].float()
        if "b1" in s:
            z = z + s["b1"].float()
    if du is not None:
        h = s["scale"] * r + (z if g is None else g * z)
        dn, hn = _norm_back(du, h, *n2, c["before"], s["w2"])
        dh = dh + dn
        out["w2"] = _rows(du * hn)
        if "b2" in s:
            out["b2"] = _rows(du)
    out["r"] = s["scale"] * dh
    dz = dh if g is None else dh * g
    if c["after"] != "none":
        out["y"], _ = _norm_back(dz, y, *n1, c["after"], s["w1"])
        out["w1"] = _rows(dz * yn)
        if "b1" in s:
            out["b1"] = _rows(dz)
    else:
        out["y"] = dz
    if g is not None:
        dims = {"channel": (0, 1), "sequence": (1,), "token": (2,)}[c["gate"]]
        out["g"] = (dh * z).sum(dims, keepdim=c["gate"] != "channel")
    return out


def _plain_join(s):
    c = s["case"]
    h, u, g, n1, n2 = _join_forward(s, s["r"].float(), s["y"].float())
    out = {"h": h.to(s["r"].dtype), "u": None if u is None else u.to(s["y"].dtype)}
    if c["train"]:
        back = _join_back(s, s["dh"].float(), s["du"].float() if "du" in s else None, _kept(s["r"], c),
                          _kept(s["y"], c), g, n1, n2)
        out.update({k: v.to(s[k].dtype) for k, v in back.items()})
    return out


_OWN = {"mx8": _own_mx8, "act": _own_act, "norm": _own_norm, "join": _own_join}
_PLAIN = {"mx8": _plain_mx8, "act": _plain_act, "norm": _plain_norm, "join": _plain_join}


# ---------------------------------------------------------------------------
# The same in 64 bits
# ---------------------------------------------------------------------------

def _times2(x, e):
    """x 2^e for float64 x, the power made from its bits."""
    return x * ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values8(x):
    """Nearest multiple of the spacing that E4M3 has at each magnitude, the largest of a group between 2^7 and 2^8."""
    rows = x.double().reshape(-1, x.shape[-1])
    cols = rows.shape[1]
    y = torch.nn.functional.pad(rows, (0, -cols % GROUP)).reshape(rows.shape[0], -1, GROUP)
    top = torch.frexp(y.abs().amax(2, keepdim=True))[1] - 1
    s = torch.clamp(top - 7, min=-126)
    a = _times2(y, -s)
    at = torch.clamp(torch.frexp(a)[1] - 1, min=-6) - 3
    return _times2(_times2(torch.round(_times2(a, -at)), at), s).reshape(rows.shape[0], -1)[:, :cols].reshape(x.shape)


def _logistic(x):
    """1 / (1 + e^-x) and its slope."""
    e = torch.exp(-x.abs())
    p = torch.where(x >= 0, 1.0, e) / (1 + e)
    return p, e / (1 + e) ** 2


def _exact_act(x, act):
    """The activation and its derivative."""
    if act == "silu":
        p, d = _logistic(x)
        return x * p, p + x * d
    if act == "gelu":
        p = torch.special.ndtr(x)
        return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(8 / math.pi)
        p, d = _logistic(k * (x + TANH_B * x ** 3))
        return x * p, p + x * d * k * (1 + 3 * TANH_B * x ** 2)
    up = (x > 0).double()
    return (x * up, up) if act == "relu" else (x * x * up, 2 * x * up)


def _exact_norm(x, kind, w, b):
    n = x.shape[-1]
    mu = x.sum(-1, keepdim=True) / n if kind == "layer" else 0.0
    sd = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / n + EPS)
    u = (x - mu) / sd * w.double()
    return (u if b is None else u + b.double()), mu, sd


def _exact_norm_back(du, kept, mu, sd, kind, w):
    """dx, dw, db: the Jacobian of x -> (x - mu) / sd at the kept values."""
    n = kept.shape[-1]
    v = (kept - mu) / sd
    g = du * w.double()
    along = (g * v).sum(-1, keepdim=True) / n
    dx = (g - v * along - (g.sum(-1, keepdim=True) / n if kind == "layer" else 0.0)) / sd
    flat = (-1, kept.shape[-1])
    return dx, (du * v).reshape(flat).sum(0), du.reshape(flat).sum(0)


def exact(case, seed):
    global own
    was, own = own, False  # inputs as plain tensors
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, low, train = case["op"], case.get("keep") == "mx8", case.get("train", False)
    keep = _exact_values8 if low else torch.Tensor.double
    if op == "mx8":
        return _exact_values8(s["x"])
    if op == "act":
        f, x = case["cols"], s["x"]
        a, b = x[:, :f], x[:, f:]
        y = _exact_act(a.double(), case["act"])[0]
        out = {"y": y * b.double() if case["gated"] else y}
        if train:
            v, d = _exact_act(keep(a), case["act"])
            dy = s["dy"].double()
            out["dx"] = torch.cat((dy * d * keep(b), dy * v), 1) if case["gated"] else dy * d
        return out
    if op == "norm":
        u, mu, sd = _exact_norm(s["x"].double(), case["kind"], s["w2"], s.get("b2"))
        out = {"u": u}
        if train:
            out["x"], out["w2"], db = _exact_norm_back(s["du"].double(), keep(s["x"]), mu, sd, case["kind"], s["w2"])
            if "b2" in s:
                out["b2"] = db
        return out
    r, y = s["r"].double(), s["y"].double()
    z = y
    if case["after"] != "none":
        z, mu1, sd1 = _exact_norm(y, case["after"], s["w1"], s.get("b1"))
    gate = s["g"].double() if "g" in s else 1.0
    h = s["scale"] * r + gate * z
    out = {"h": h, "u": None}
    if case["before"] != "none":
        out["u"], mu2, sd2 = _exact_norm(h, case["before"], s["w2"], s.get("b2"))
    if not train:
        return out
    total, ky = s["dh"].double(), keep(s["y"])
    kz = ky
    if case["after"] != "none":
        kz = (ky - mu1) / sd1 * s["w1"].double()
        if "b1" in s:
            kz = kz + s["b1"].double()
    if "du" in s:
        kh = s["scale"] * keep(s["r"]) + gate * kz
        dx, out["w2"], db = _exact_norm_back(s["du"].double(), kh, mu2, sd2, case["before"], s["w2"])
        total = total + dx
        if "b2" in s:
            out["b2"] = db
    out["r"] = s["scale"] * total
    out["y"] = dz = total * gate
    if case["after"] != "none":
        out["y"], out["w1"], db = _exact_norm_back(dz, ky, mu1, sd1, case["after"], s["w1"])
        if "b1" in s:
            out["b1"] = db
    if case["gate"] == "channel":
        out["g"] = (total * kz).sum((0, 1))
    elif case["gate"] == "sequence":
        out["g"] = (total * kz).sum(1, keepdim=True)
    elif case["gate"] == "token":
        out["g"] = (total * kz).sum(2, keepdim=True)
    return out
