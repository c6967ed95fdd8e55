"""Norms and joins against the float64 oracle, forward and backward."""
import itertools
import math

import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from oracle import layers_oracle as O
from layers_helpers import check, normal, strided

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (F32, BF16), (BF16, BF16)]

# Roundings on the way to a result.  A sum over a row adds at most 32 elements in
# a lane, 6 levels of a wave and 8 waves: 46, and a norm has two sums in a row
# (mean, variance) that meet a result: 100 with the element's own operations.  h
# and u see two norms, a gradient both norms again and its own two pairs of sums.
# A column's sum adds at most 32 rows here, then 48 partial ones.
FORWARD, BACKWARD = 256, 512


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _norms(gen, kind, cols, bias, param, weight=True):
    if kind is None:
        return None, None
    w = normal(gen, cols, dtype=param, std=0.2) + 1 if weight else None
    b = normal(gen, cols, dtype=param, std=0.3) if bias else None
    return L.Norm(kind, w, b, 1e-5), (kind, None if w is None else w.cpu(), None if b is None else b.cpu(),
                                      float(torch.tensor(1e-5)))


def _require(*tensors):
    for t in tensors:
        if t is not None:
            t.requires_grad_()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("types", TYPES, ids=["f32", "mixed", "bf16"])
@pytest.mark.parametrize("keep", ["same", "mx8"])
@pytest.mark.parametrize("cols", [1, 3, 8, 33, 250, 257, 512, 700, 1024, 1025, 2048, 2050, 4096, 4100, 8192, 9001, 16384])
def test_norm(kind, types, keep, cols):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    for rows, bias, layout in ((1, False, "plain"), (3, True, "padded"), (70 if cols < 3000 else 9, True, "plain")):
        x = strided((normal(gen, rows, cols, std=2.0) + (0.5 if cols > 1 else 0)).to(types[0]), layout)
        n, ref = _norms(gen, kind, cols, bias, F32 if rows > 1 else BF16)
        _require(x, n.weight, n.bias)
        u = L.norm(x, n, dtype=types[1], keep=keep)
        xd = x.detach().cpu()
        o, m = (O.join(xd, None, n2=ref, magnitude=k) for k in (False, True))
        name = f"{rows} rows {layout} "
        check(u, o.u, m.u, FORWARD, name + "u")
        du = strided(normal(gen, rows, cols, dtype=types[1]), layout)
        leaves = [t for t in (x, n.weight, n.bias) if t is not None]
        got = torch.autograd.grad(u, leaves, du)
        want, mag = (O.join_backward(O.kept(xd, keep), None, None, o.st2, n2=ref, du=du.cpu(), magnitude=k)
                     for k in (False, True))
        for g, w in zip(got, ("r", "w2", "b2")):
            check(g, getattr(want, w), getattr(mag, w), BACKWARD, name + w)
        with torch.no_grad():
            assert torch.equal(L.norm(x, n, dtype=types[1]), u)


def _join_case(gen, seqs, length, cols, after, before, gate, bias, types, param, layout="plain"):
    shape = (seqs, length, cols)
    r = strided(normal(gen, *shape, dtype=types[0], std=2.0), layout)
    y = strided(normal(gen, *shape, dtype=types[1], std=0.5), layout)
    n1, ref1 = _norms(gen, after, cols, bias, param)
    n2, ref2 = _norms(gen, before, cols, bias, param)
    size = {"channel": (cols,), "sequence": (seqs, 1, cols), "token": (seqs, length, 1), "row": shape}.get(gate)
    g = None if gate is None else (normal(gen, *size, std=0.5) + 0.5).to(param)
    leaves = {"r": r, "y": y, "w1": n1 and n1.weight, "b1": n1 and n1.bias, "gate": g, "w2": n2 and n2.weight,
              "b2": n2 and n2.bias}
    leaves = {k: t for k, t in leaves.items() if t is not None}
    _require(*leaves.values())
    return r, y, n1, n2, g, ref1, ref2, leaves


def _check_join(case, keep, scale, dh, du, name=""):
    r, y, n1, n2, g, ref1, ref2, leaves = case
    h, u = L.join(r, y, after=n1, gate=g, scale=scale, before=n2, keep=keep)
    rd, yd, gd = r.detach().cpu(), y.detach().cpu(), None if g is None else g.detach().cpu()
    s32 = float(torch.tensor(scale))
    o, m = (O.join(rd, yd, ref1, gd, s32, ref2, magnitude=k) for k in (False, True))
    assert h.dtype == r.dtype and h.shape == r.shape
    check(h, o.h, m.h, FORWARD, name + " h")
    outs, grads = [], []
    if n2 is None:
        assert u is None
    else:
        assert u.dtype == y.dtype
        check(u, o.u, m.u, FORWARD, name + " u")
    if dh is not None:
        outs.append(h), grads.append(dh)
    if n2 is not None and du is not None:
        outs.append(u), grads.append(du)
    if not outs:
        return h, u
    got = dict(zip(leaves, torch.autograd.grad(outs, list(leaves.values()), grads, allow_unused=True)))
    want, mag = (O.join_backward(O.kept(rd, keep), O.kept(yd, keep), o.st1, o.st2, ref1, gd, s32, ref2,
                                 None if dh is None else dh.cpu(), du.cpu() if n2 is not None and du is not None else None,
                                 magnitude=k) for k in (False, True))
    for k, v in got.items():
        if v is None:
            assert getattr(want, k) is None, (name, k)
        else:
            check(v, getattr(want, k), getattr(mag, k), BACKWARD, f"{name} d{k}")
    return h, u


@pytest.mark.parametrize("after", [None, "rms", "layer"])
@pytest.mark.parametrize("before", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "channel", "sequence", "token", "row"])
@pytest.mark.parametrize("keep", ["same", "mx8"])
def test_join_of_every_form(after, before, gate, keep):
    gen = torch.Generator(device="cuda").manual_seed(11)
    for types, bias, param, layout in zip(TYPES, (True, False, True), (F32, BF16, BF16), ("plain", "padded", "plain")):
        for seqs, length, cols in ((2, 3, 65), (3, 7, 520)):
            case = _join_case(gen, seqs, length, cols, after, before, gate, bias, types, param, layout)
            dh = normal(gen, seqs, length, cols, dtype=types[0])
            du = normal(gen, seqs, length, cols, dtype=types[1])
            _check_join(case, keep, 0.75, dh, du, f"{types} {cols}")


@pytest.mark.parametrize("types", TYPES, ids=["f32", "mixed", "bf16"])
@pytest.mark.parametrize("cols", [1, 7, 256, 511, 513, 1024, 1500, 2048, 2051, 4096, 5000, 8192, 8200, 16384])
def test_join_of_every_width(types, cols):
    gen = torch.Generator(device="cuda").manual_seed(cols + 1)
    seqs, length = (1, 1) if cols % 2 else (2, 5)
    for keep, bias, gate in (("same", True, "channel"), ("mx8", False, "sequence"), ("same", False, "token"),
                             ("mx8", True, "channel")):
        case = _join_case(gen, seqs, length, cols, "rms", "layer", gate, bias, types, F32)
        _check_join(case, keep, 1.0, normal(gen, seqs, length, cols, dtype=types[0]),
                    normal(gen, seqs, length, cols, dtype=types[1]), f"{keep} {gate}")


@pytest.mark.parametrize("gate,seqs,length", [("channel", 1, 3000), ("sequence", 1, 1500), ("sequence", 5, 700),
                                              ("sequence", 1000, 3), ("sequence", 4000, 1), ("row", 40, 50),
                                              ("token", 30, 100), ("sequence", 37, 61)])
@pytest.mark.parametrize("keep", ["same", "mx8"])
def test_sums_over_many_rows(gate, seqs, length, keep):
    """Rows spread over many workgroups, in runs longer and shorter than a workgroup's share."""
    gen = torch.Generator(device="cuda").manual_seed(seqs)
    case = _join_case(gen, seqs, length, 48, "layer", "rms", gate, True, (F32, F32), F32)
    _check_join(case, keep, 0.5, normal(gen, seqs, length, 48), normal(gen, seqs, length, 48))


@pytest.mark.parametrize("types", TYPES, ids=["f32", "mixed", "bf16"])
@pytest.mark.parametrize("gate,seqs,length,cols", [("channel", 1, 700, 9000), ("sequence", 2, 280, 8203),
                                                   ("row", 30, 20, 9001), (None, 3, 180, 16384)])
@pytest.mark.parametrize("bias", [False, True])
def test_sums_of_wide_rows(types, gate, seqs, length, cols, bias):
    """Workgroups that take some rows each of more than 8192 columns."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    case = _join_case(gen, seqs, length, cols, "rms", "layer", gate, bias, types, F32)
    _check_join(case, "mx8" if seqs % 2 else "same", 1.0, normal(gen, seqs, length, cols, dtype=types[0]),
                normal(gen, seqs, length, cols, dtype=types[1]))


@pytest.mark.parametrize("given", ["h", "u"])
@pytest.mark.parametrize("keep", ["same", "mx8"])
def test_a_gradient_of_one_output_only(given, keep):
    gen = torch.Generator(device="cuda").manual_seed(5)
    for after, gate in itertools.product((None, "rms"), (None, "channel", "token")):
        case = _join_case(gen, 2, 9, 100, after, "layer", gate, True, (F32, F32), F32)
        dh, du = normal(gen, 2, 9, 100), normal(gen, 2, 9, 100)
        _check_join(case, keep, 1.0, dh if given == "h" else None, du if given == "u" else None)


def test_only_some_inputs_need_gradients():
    gen = torch.Generator(device="cuda").manual_seed(6)
    names = ("r", "y", "w1", "b1", "gate", "w2", "b2")
    for keep in ("same", "mx8"):
        r, y, n1, n2, g, ref1, ref2, leaves = _join_case(gen, 2, 30, 100, "layer", "layer", "sequence", True, (F32, F32), F32)
        dh, du = normal(gen, 2, 30, 100), normal(gen, 2, 30, 100)
        h, u = L.join(r, y, n1, g, 0.5, n2, keep)
        want = dict(zip(leaves, torch.autograd.grad((h, u), list(leaves.values()), (dh, du))))
        for some in ((k,) for k in names):
            for k, t in leaves.items():
                t.requires_grad_(k in some)
            h, u = L.join(r, y, n1, g, 0.5, n2, keep)
            for k, got in zip(some, torch.autograd.grad((h, u), [leaves[k] for k in some], (dh, du))):
                assert torch.equal(got, want[k]), k


def test_gradients_against_differences():
    gen = torch.Generator(device="cuda").manual_seed(8)
    r, y, n1, n2, g, ref1, ref2, leaves = _join_case(gen, 2, 3, 40, "layer", "rms", "sequence", True, (F32, F32), F32)
    dh, du = normal(gen, 2, 3, 40), normal(gen, 2, 3, 40)
    h, u = L.join(r, y, n1, g, 0.5, n2)
    grads = torch.autograd.grad((h, u), list(leaves.values()), (dh, du))

    def loss():
        with torch.no_grad():
            h, u = L.join(r, y, n1, g, 0.5, n2)
            return (h.double() * dh).sum() + (u.double() * du).sum()
    step = 2.0 ** -9
    for t, grad in zip(leaves.values(), grads):
        d = normal(gen, *t.shape)
        with torch.no_grad():
            t += step * d
            up = loss()
            t -= 2 * step * d
            down = loss()
            t += step * d
        # 240 outputs of error 2^-20 weighted by normal numbers, over 2^-8; third order (step^2) terms of 240 of them
        tol = 6 * 240 ** 0.5 * 2.0 ** -20 / 2 ** -8 + 240 * step ** 2 * 8
        assert abs((up - down).item() / (2 * step) - (grad.double() * d).sum().item()) <= tol


def test_weights_may_be_missing():
    gen = torch.Generator(device="cuda").manual_seed(9)
    for kind, cols in itertools.product(("rms", "layer"), (5, 100, 1030)):
        x = normal(gen, 6, cols) + 1
        n, ref = _norms(gen, kind, cols, False, F32, weight=False)
        x.requires_grad_()
        u = L.norm(x, n)
        o, m = (O.join(x.detach().cpu(), None, n2=ref, magnitude=k) for k in (False, True))
        check(u, o.u, m.u, FORWARD, kind)
        y = normal(gen, 6, cols).requires_grad_()
        g = normal(gen, cols).requires_grad_()
        h, u = L.join(x, y, n, g, 1.0, n)
        o, m = (O.join(x.detach().cpu(), y.detach().cpu(), ref, g.detach().cpu(), 1.0, ref, magnitude=k) for k in (False, True))
        check(h, o.h, m.h, FORWARD, kind)
        check(u, o.u, m.u, FORWARD, kind)
        dh, du = normal(gen, 6, cols), normal(gen, 6, cols)
        got = torch.autograd.grad((h, u), (x, y, g), (dh, du))
        want, mag = (O.join_backward(x.detach().cpu(), y.detach().cpu(), o.st1 if o.st1 else None, o.st2, ref,
                                     g.detach().cpu(), 1.0, ref, dh.cpu(), du.cpu(), magnitude=k)
                     for o, k in ((O.join(x.detach().cpu(), y.detach().cpu(), ref, g.detach().cpu(), 1.0, ref), k)
                                  for k in (False, True)))
        for v, k in zip(got, ("r", "y", "gate")):
            check(v, getattr(want, k), getattr(mag, k), BACKWARD, k)


def test_rows_of_zeros_and_special_rows():
    """A padded row (all zero) is finite; NaN and infinities stay in their rows and, of gradients, in their columns' sums."""
    gen = torch.Generator(device="cuda").manual_seed(10)
    for kind, keep in itertools.product(("rms", "layer"), ("same", "mx8")):
        x = normal(gen, 9, 300)
        x[2], x[5, 7], x[6, 9] = 0, math.nan, math.inf
        n, ref = _norms(gen, kind, 300, True, F32)
        _require(x, n.weight, n.bias)
        u = L.norm(x, n, keep=keep)
        dx, dw, db = torch.autograd.grad(u, (x, n.weight, n.bias), torch.ones_like(u))
        ok = [0, 1, 2, 3, 4, 7, 8]
        assert torch.isfinite(u[ok]).all() and torch.isfinite(dx[ok]).all() and torch.isfinite(db).all()
        assert torch.isnan(u[5]).all() and torch.isnan(u[6]).any()
        assert torch.equal(u[2], n.bias)
        clean = x.detach()[ok].requires_grad_()
        assert torch.equal(L.norm(clean, n, keep=keep), u[ok])
        got, = torch.autograd.grad(L.norm(clean, n, keep=keep), clean, torch.ones(7, 300, device="cuda"))
        assert torch.equal(got, dx[ok])


def test_layernorm_of_a_large_mean():
    """The variance is taken about the mean: 1000 +- 1 keeps 14 bits of the difference."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = 1000 + normal(gen, 5, 777)
    n = L.Norm("layer", eps=1e-5)
    o = O.join(x.cpu(), None, n2=("layer", None, None, float(torch.tensor(1e-5))))
    # x is exact; the mean's error (46 roundings of 1000) moves every element by 46 * 1000 * 2^-24 at most
    assert (L.norm(x, n).cpu().double() - o.u).abs().max() <= 46 * 1000 * 2.0 ** -24 * 1.1 + 64 * 2.0 ** -24 * 5


def test_the_same_tensor_twice():
    """Residual and branch one tensor, one weight for both norms: gradients add up."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    x = normal(gen, 20, 130).requires_grad_()
    w = (normal(gen, 130) * 0.1 + 1).requires_grad_()
    n = L.Norm("rms", w)
    h, u = L.join(x, x, after=n, before=n)
    dx, dw = torch.autograd.grad((h, u), (x, w), (torch.ones_like(h), torch.ones_like(u)))
    a, b = x.detach().clone().requires_grad_(), x.detach().clone().requires_grad_()
    w1, w2 = w.detach().clone().requires_grad_(), w.detach().clone().requires_grad_()
    h2, u2 = L.join(a, b, after=L.Norm("rms", w1), before=L.Norm("rms", w2))
    ga, gb, g1, g2 = torch.autograd.grad((h2, u2), (a, b, w1, w2), (torch.ones_like(h), torch.ones_like(u)))
    assert torch.equal(h, h2) and torch.equal(u, u2)
    assert torch.equal(dx, ga + gb) and torch.equal(dw, g1 + g2)


def test_rows_beyond_32_bit_offsets():
    rows, cols = (1 << 18) + 70, 8192
    x = torch.zeros(rows, cols, device="cuda", dtype=BF16)
    gen = torch.Generator(device="cuda").manual_seed(14)
    tail = normal(gen, 6, cols, dtype=BF16)
    x[-6:] = tail
    n = L.Norm("rms", torch.ones(cols, device="cuda").requires_grad_())
    x.requires_grad_()
    u = L.norm(x, n, keep="mx8")
    t = tail.clone().requires_grad_()
    v = L.norm(t, n, keep="mx8")
    assert torch.equal(u[-6:], v)
    dv = normal(gen, 6, cols, dtype=BF16)
    du = torch.zeros_like(u)
    du[-6:] = dv
    dx, dw = torch.autograd.grad(u, (x, n.weight), du)
    dt, dw2 = torch.autograd.grad(v, (t, n.weight), dv)
    assert torch.equal(dx[-6:], dt) and not dx[:1000].any()
    assert torch.allclose(dw, dw2, rtol=1e-5, atol=1e-5)


def test_repeated_calls_give_the_same_bits():
    gen = torch.Generator(device="cuda").manual_seed(15)
    case = _join_case(gen, 8, 300, 700, "rms", "rms", "sequence", True, (BF16, BF16), F32)
    r, y, n1, n2, g, _, _, leaves = case
    dh, du = normal(gen, 8, 300, 700, dtype=BF16), normal(gen, 8, 300, 700, dtype=BF16)
    runs = []
    for _ in range(3):
        h, u = L.join(r, y, n1, g, 1.0, n2, "mx8")
        runs.append([h.detach(), u.detach(), *torch.autograd.grad((h, u), list(leaves.values()), (dh, du))])
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_empty():
    n = L.Norm("rms", torch.ones(6, device="cuda", requires_grad=True), torch.zeros(6, device="cuda", requires_grad=True))
    x = torch.zeros(0, 6, device="cuda", requires_grad=True)
    g = torch.ones(6, device="cuda", requires_grad=True)
    for keep in ("same", "mx8"):
        dx, dw, db = torch.autograd.grad(L.norm(x, n, keep=keep).sum(), (x, n.weight, n.bias))
        assert dx.shape == (0, 6) and not dw.any() and not db.any()
        h, u = L.join(x, x.detach(), n, g, 1.0, n, keep)
        dx, dw, dg = torch.autograd.grad(h.sum() + u.sum(), (x, n.weight, g))
        assert dx.shape == (0, 6) and not dw.any() and not dg.any()
    e = torch.zeros(4, 0, device="cuda")
    assert L.norm(e, L.Norm()).shape == (4, 0)


def test_refusals():
    x, y = torch.randn(2, 3, 64, device="cuda"), torch.randn(2, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    n = L.Norm("rms", w)
    wide = torch.zeros(2, capi.NORM_COLS + 1, device="cuda")
    for bad in (lambda: L.Norm("batch"), lambda: L.Norm(eps=0.0), lambda: L.Norm(eps=math.nan), lambda: L.norm(x, None),
                lambda: L.norm(x, w), lambda: L.norm(x.half(), n), lambda: L.norm(x.cpu(), n),
                lambda: L.norm(x.bfloat16(), n, dtype=F32), lambda: L.norm(x, n, dtype=torch.float16),
                lambda: L.norm(x, L.Norm("rms", w[:63])), lambda: L.norm(x, L.Norm("rms", w.half())),
                lambda: L.norm(x, L.Norm("rms", w.cpu())), lambda: L.norm(x, L.Norm("rms", w[None])),
                lambda: L.norm(x, n, keep="mx4"), lambda: L.join(x, y[:1], before=n), lambda: L.join(x.bfloat16(), y),
                lambda: L.join(x, y, gate=w[:32]), lambda: L.join(x, y, gate=torch.ones(3, 1, 64, device="cuda")),
                lambda: L.join(x, y, gate=torch.ones(1, 3, 64, device="cuda")), lambda: L.join(x, y, gate=w.cpu()),
                lambda: L.join(x, y, gate=w.half()), lambda: L.join(x, y, scale=math.inf), lambda: L.join(x, y, after=w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(capi.ShampooError):
        L.norm(wide, L.Norm())
