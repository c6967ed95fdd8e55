"""Activations and gated activations against the float64 oracle, forward and
backward, with their inputs kept as they are and in MX8."""
import itertools
import math

import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from oracle import layers_oracle as O
from layers_helpers import HALF, check, normal, strided

pytestmark = pytest.mark.gpu

# fp32 roundings that reach a result: an exponential (3, its argument in two floats),
# a reciprocal, a polynomial (7: 4.1e-7 on all of its range, measured in fp32 arithmetic,
# its fit included), products.  16 cover them; with derivative and gate 24.  For
# bf16 results the argument is one float: up to 112, after 4 roundings, so that the exponential
# is off by 4 * 112 * 1.44 more.
FORWARD = {torch.float32: 16, torch.bfloat16: 16 + 650}
BACKWARD = {torch.float32: 24, torch.bfloat16: 24 + 2 * 650}
# The exponential is 0 below 2^-126.  It is multiplied by x (12 here and 2^6 at most where it is
# that small), for the slope by x v', at most 12 * 31 (tanh), and by the gradients, below 2^3.
LEAST = 2.0 ** -114


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _slope_magnitude(x, f, d):
    """Of the two terms p and x p' whose sum is the slope."""
    p = torch.where(x == 0, d, f / torch.where(x == 0, 1.0, x)).abs()
    return p + (d - p).abs()


def _inputs(rows, cols, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    a = normal(gen, rows, cols, std=3.0)
    a.view(-1)[::7] *= 4                       # into the tails
    return a.to(dtype), normal(gen, rows, cols, dtype=dtype), normal(gen, rows, cols, dtype=dtype)


SIZES = [(1, 1), (1, 5), (3, 31), (2, 33), (1, 2048), (67, 100), (130, 515), (33, 4104)]


@pytest.mark.parametrize("act", O.ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("keep", ["same", "mx8"])
@pytest.mark.parametrize("form", ["plain", "gated", "packed"])
def test_values_and_gradients(act, dtype, keep, form):
    for (rows, cols), layout in itertools.product(SIZES, ("plain", "padded")):
        a, b, dy = _inputs(rows, cols, dtype, rows + cols)
        name = f"{rows}x{cols} {layout}"
        if form == "packed":
            x = strided(torch.cat((a, b), 1), layout).requires_grad_()
            y = L.gated(x, act=act, keep=keep)
            da, db = torch.autograd.grad(y, x, dy)[0].split(cols, 1)
        elif form == "gated":
            a_, b_ = strided(a, layout).requires_grad_(), strided(b, layout).requires_grad_()
            y = L.gated(a_, b_, act=act, keep=keep)
            da, db = torch.autograd.grad(y, (a_, b_), strided(dy, layout))
        else:
            a_ = strided(a, layout).requires_grad_()
            y = L.activation(a_, act=act, keep=keep)
            da, = torch.autograd.grad(y, a_, strided(dy, layout))
        gate = form != "plain"
        f, _ = O.act(a.cpu(), act)
        bd = b.cpu().double() if gate else torch.ones_like(f)
        check(y, f * bd, (f * bd).abs(), FORWARD[dtype], name, LEAST)
        with torch.no_grad():
            again = (L.activation(a, act=act) if not gate else L.gated(a, b, act=act))
        assert torch.equal(again, y)
        ak, bk = O.kept(a.cpu(), keep), O.kept(b.cpu(), keep) if gate else bd
        f, d = O.act(ak, act)
        g = dy.cpu().double()
        check(da, g * d * bk, (g * bk).abs() * _slope_magnitude(ak, f, d), BACKWARD[dtype], name + " da", LEAST)
        if gate:
            check(db, g * f, (g * f).abs(), BACKWARD[dtype], name + " db", LEAST)


@pytest.mark.parametrize("act", O.ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_and_special_values(act, dtype):
    """Values of every binade; 0 and 1 slopes far out; infinities and NaN as in the formulas' limits."""
    e = torch.arange(-126, 127, dtype=torch.float64)
    x = torch.cat((2.0 ** e, -2.0 ** e, 1.7 * 2.0 ** e, -1.7 * 2.0 ** e, torch.linspace(-130, 130, 5001).double(),
                   torch.zeros(1, dtype=torch.float64)))
    x = x.to(dtype).cuda()[None].requires_grad_()
    y = L.activation(x, act=act)
    dx, = torch.autograd.grad(y, x, torch.ones_like(y))
    f, d = O.act(x.detach().cpu(), act)
    limit = torch.finfo(dtype).max
    f = torch.where(f.abs() > limit * (1 + HALF[dtype]), math.inf, f)
    check(y, f, torch.nan_to_num(f.abs(), posinf=0.0), FORWARD[dtype], least=LEAST)
    d = torch.where(d.abs() > limit * (1 + HALF[dtype]), math.inf, d)
    check(dx, d, torch.nan_to_num(_slope_magnitude(x.detach().cpu().double(), f, d), nan=1.0, posinf=0.0), BACKWARD[dtype], least=LEAST)
    s = torch.tensor([[math.inf, math.nan]], device="cuda", dtype=dtype).requires_grad_()
    y = L.activation(s, act=act)
    dx, = torch.autograd.grad(y, s, torch.ones_like(y))
    assert y[0, 0] == math.inf and torch.isnan(y[0, 1])
    assert dx[0, 0] == (math.inf if act == "relu2" else 1.0)
    assert torch.isnan(dx[0, 1])


def test_gelu_keeps_the_tail():
    x = torch.linspace(-12, 0, 20001, device="cuda")[None]
    want = O.act(x.cpu(), "gelu")[0]
    off = (L.activation(x, act="gelu").cpu().double() / want - 1).abs()[0, :-1]
    assert off.max() <= FORWARD[torch.float32] * 2.0 ** -24


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu2"])
def test_gradients_against_differences(act):
    """dy . (f(x + h) - f(x - h)) b / 2h in float64 of the kernel's own formula's oracle, and by the kernel."""
    a, b, dy = _inputs(5, 70, torch.float32, 3)
    a, h = a.clamp(-4, 4).requires_grad_(), 2.0 ** -7
    y = L.gated(a, b, act=act)
    da, = torch.autograd.grad(y, a, dy)
    with torch.no_grad():
        diff = (L.gated(a + h, b, act=act) - L.gated(a - h, b, act=act)) / (2 * h)
    # third derivatives are below 4 (relu2: a kink of curvature 2 across h), rounding 2^-22 |y| / h
    tol = dy.abs() * (b.abs() * (4 * h * h / 6 + (h if act == "relu2" else 0)) + 2.0 ** -21 * (y.abs() + b.abs()) / h)
    assert ((da - dy * diff).abs() <= tol).all()


def test_only_what_is_needed():
    a, b, dy = _inputs(9, 70, torch.float32, 5)
    for need in ((True, False), (False, True)):
        for keep in ("same", "mx8"):
            aa, bb = a.clone().requires_grad_(need[0]), b.clone().requires_grad_(need[1])
            y = L.gated(aa, bb, act="silu", keep=keep)
            got, = torch.autograd.grad(y, aa if need[0] else bb, dy)
            assert got.shape == a.shape
            ak, bk = O.kept(a.cpu(), keep), O.kept(b.cpu(), keep)
            f, d = O.act(ak, "silu")
            want = dy.cpu().double() * (d * bk if need[0] else f)
            check(got, want, want.abs() + (dy.cpu() * b.cpu()).abs().double(), BACKWARD[torch.float32])


def test_shapes_strides_and_expanded_gradients():
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = normal(gen, 3, 5, 4, 64)
    cases = {"transposed": x.transpose(0, 2), "sliced": x[:, 1:4], "columns apart": strided(x, "apart"),
             "negated view": torch.view_as_complex(normal(gen, 5, 64, 2)).conj().imag, "one dimension": x[0, 0, 0],
             "padded": strided(x, "padded"), "expanded": x[:1].expand(3, 5, 4, 64)}
    for name, t in cases.items():
        want = L.activation(t.contiguous())
        assert torch.equal(L.activation(t), want), name
        leaf = t.detach().requires_grad_()
        y = L.activation(leaf)
        dx, = torch.autograd.grad(y.sum(), leaf)                 # an expanded gradient
        c = t.contiguous().requires_grad_()
        assert torch.equal(dx, torch.autograd.grad(L.activation(c), c, torch.ones_like(c))[0]), name


def test_empty():
    for shape in ((0, 6), (6, 0), (0,)):
        for keep in ("same", "mx8"):
            x = torch.zeros(shape, device="cuda", requires_grad=True)
            for y in (L.activation(x, keep=keep), L.gated(x, keep=keep), L.gated(x, x.detach(), keep=keep)):
                assert torch.autograd.grad(y.sum(), x)[0].shape == x.shape


def test_refusals():
    x = torch.randn(4, 64, device="cuda")
    for bad in (lambda: L.activation(x, act="tanh"), lambda: L.activation(x, keep="mx4"), lambda: L.activation(x.half()),
                lambda: L.activation(x.cpu()), lambda: L.gated(x[:, :63]), lambda: L.gated(x, x[:2]),
                lambda: L.gated(x, x.bfloat16()), lambda: L.activation(x.sum())):
        with pytest.raises(ValueError):
            bad()
