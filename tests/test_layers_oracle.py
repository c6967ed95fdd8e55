"""Pins of the float64 oracle of the layers: E4M3's table, torch's own float64
functions, autograd and differences."""
import math

import pytest
import torch

from oracle import layers_oracle as O

F = torch.nn.functional


def _gen(seed=0):
    return torch.Generator().manual_seed(seed)


def test_codes_are_ocp_e4m3_rounded_to_nearest_even():
    """A group whose largest is 128 has s = 127, so that codes stand for themselves."""
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    x = torch.linspace(-131, 131, 100001, dtype=torch.float64)
    near = table[torch.isfinite(table)].unique()
    ties = (near[1:] + near[:-1]) / 2
    x = torch.cat((x, near, ties, ties * (1 + 2 ** -40)))
    x = x[x.abs() < 255]
    x = F.pad(x, (0, -x.numel() % 31)).reshape(-1, 31)
    x = torch.cat((x, torch.full((x.shape[0], 1), 128.0, dtype=torch.float64)), 1)
    codes, s = O.mx8_codes(x)
    # float8 rounds from float32: values whose float32 is the same rounding
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).long()
    exact = x.float().double() == x
    assert (s == 127).all() and (codes == want)[exact].all()
    value = O.mx8_decode(codes, s, 32)
    assert torch.equal(value, table[codes])
    d = (value - x).abs()
    assert (d <= torch.clamp(2.0 ** -4 * x.abs(), min=2.0 ** -10)).all()


def test_scales_of_special_groups():
    rows = torch.zeros(6, 32, dtype=torch.float64)
    rows[1, 3] = math.inf
    rows[2, 5] = math.nan
    rows[3, 0] = 2.0 ** -149
    rows[4, 31] = torch.finfo(torch.float32).max
    rows[5] = -0.0
    codes, s = O.mx8_codes(rows)
    assert s[:, 0].tolist() == [1, 255, 255, 1, 247, 1]
    v = O.mx8_decode(codes, s, 32)
    assert torch.isnan(v[1:3]).all() and (v[0] == 0).all() and (v[3] == 0).all()
    assert v[4, 31] == 2.0 ** 128 and (v[5] == 0).all()


@pytest.mark.parametrize("name,ref", [("silu", F.silu), ("gelu", F.gelu), ("relu", F.relu),
                                      ("gelu_tanh", lambda x: F.gelu(x, approximate="tanh")),
                                      ("relu2", lambda x: F.relu(x) ** 2)])
def test_activations_and_slopes(name, ref):
    x = torch.linspace(-9, 9, 4000, dtype=torch.float64, requires_grad=True)
    y = ref(x)
    f, d = O.act(x.detach(), name)
    assert torch.allclose(f, y.detach(), rtol=1e-12, atol=1e-13)
    assert torch.allclose(d, torch.autograd.grad(y.sum(), x)[0], rtol=1e-11, atol=1e-12)


def _case(after, before, gate, bias=True, seqs=3, n=5, cols=37):
    gen = _gen(7)

    def t(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)
    p = {"r": t(seqs, n, cols), "y": t(seqs, n, cols)}
    n1 = n2 = None
    if after:
        n1 = (after, 1 + 0.2 * t(cols), 0.3 * t(cols) if bias else None, 1e-2)
    if before:
        n2 = (before, 1 + 0.2 * t(cols), 0.3 * t(cols) if bias else None, 1e-2)
    shape = {"channel": (cols,), "sequence": (seqs, 1, cols), "token": (seqs, n, 1)}.get(gate)
    g = t(*shape) if gate else None
    return p, n1, n2, g, t


@pytest.mark.parametrize("after", [None, "rms", "layer"])
@pytest.mark.parametrize("before", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "channel", "sequence", "token"])
def test_join_and_its_gradients(after, before, gate):
    p, n1, n2, g, t = _case(after, before, gate)
    leaves = {"r": p["r"], "y": p["y"], "gate": g}
    for tag, n in (("1", n1), ("2", n2)):
        leaves["w" + tag], leaves["b" + tag] = (n[1], n[2]) if n else (None, None)
    leaves = {k: v.requires_grad_() for k, v in leaves.items() if v is not None}

    def normed(x, n):
        if n is None:
            return x
        if n[0] == "layer":
            return F.layer_norm(x, x.shape[-1:], n[1], n[2], n[3])
        return F.rms_norm(x, x.shape[-1:], n[1], n[3]) + n[2]
    z = normed(p["y"], n1)
    h = 0.75 * p["r"] + (z if g is None else g * z)
    u = normed(h, n2) if n2 else None
    o = O.join(p["r"].detach(), p["y"].detach(), n1, g, 0.75, n2)
    assert torch.allclose(o.h, h, atol=1e-12)
    dh, du = t(*h.shape), t(*h.shape)
    loss = (h * dh).sum()
    if u is not None:
        assert torch.allclose(o.u, u, atol=1e-12)
        loss = loss + (u * du).sum()
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    got = O.join_backward(p["r"], p["y"], o.st1, o.st2, n1, g, 0.75, n2, dh, du if n2 else None)
    for k, v in want.items():
        assert torch.allclose(getattr(got, k), v, atol=1e-10), k


def test_join_gradients_against_differences():
    p, n1, n2, g, t = _case("layer", "rms", "sequence")
    dh, du = t(*p["r"].shape), t(*p["r"].shape)

    def loss(r, y, gate):
        o = O.join(r, y, n1, gate, 0.75, n2)
        return ((o.h * dh).sum() + (o.u * du).sum()).item()
    o = O.join(p["r"], p["y"], n1, g, 0.75, n2)
    got = O.join_backward(p["r"], p["y"], o.st1, o.st2, n1, g, 0.75, n2, dh, du)
    step = 1e-6
    for i, grad in enumerate((got.r, got.y, got.gate)):
        d = t(*grad.shape)
        args = [p["r"], p["y"], g]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        diff = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(diff - (grad * d).sum().item()) <= 1e-7 * (1 + abs(diff))


def test_magnitudes_are_above_the_values():
    p, n1, n2, g, t = _case("layer", "layer", "channel")
    dh, du = t(*p["r"].shape), t(*p["r"].shape)
    o, m = (O.join(p["r"], p["y"], n1, g, -0.75, n2, magnitude=k) for k in (False, True))
    assert (m.h >= o.h.abs() - 1e-12).all() and (m.u >= o.u.abs() - 1e-12).all()
    a, b = (O.join_backward(p["r"], p["y"], o.st1, o.st2, n1, g, -0.75, n2, dh, du, magnitude=k) for k in (False, True))
    for k, v in vars(a).items():
        assert (getattr(b, k) >= v.abs() - 1e-12).all(), k
