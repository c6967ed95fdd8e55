"""The layers as a training step and a server use them: a block of norm, linear,
gated activation, linear and join; graphs, streams, checkpoints and what is held
until the backward pass."""
import gc
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch
from torch.autograd import forward_ad

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from inverse_root_preconditioning_amd import mx4 as MX
from inverse_root_preconditioning_amd import mx8 as M8
from oracle import layers_oracle as O
from layers_helpers import normal

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


class Blocks:
    """Two blocks h, u = join(h, down(gated(up(u)))), normed before and after."""

    def __init__(self, width, hidden, dtype=BF16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w0 = torch.ones(width, device="cuda")
        self.up = [normal(gen, 2 * hidden, width, std=width ** -0.5) for _ in range(2)]
        self.down = [normal(gen, width, hidden, std=hidden ** -0.5) for _ in range(2)]
        self.after = [1 + normal(gen, width, std=0.1) for _ in range(2)]
        self.before = [1 + normal(gen, width, std=0.1) for _ in range(2)]
        self.gate = [0.5 + normal(gen, width, std=0.1) for _ in range(2)]
        for p in self.parameters():
            p.requires_grad_()

    def parameters(self):
        return [self.w0, *self.up, *self.down, *self.after, *self.before, *self.gate]

    def forward(self, x, keep, linear=MX.train_linear):
        h, u = x, L.norm(x, L.Norm("rms", self.w0), keep=keep)
        for i in range(2):
            y = linear(L.gated(linear(u, self.up[i]), act="silu", keep=keep), self.down[i])
            h, u = L.join(h, y, after=L.Norm("rms", self.after[i]), gate=self.gate[i], before=L.Norm("rms", self.before[i]),
                          keep=keep)
        return u


def _plain_forward(net, x, linear):
    """The same from torch's elementary operations in float64."""
    def normed(t, w):
        return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
    p = [t.detach().cpu().double().requires_grad_() for t in net.parameters()]
    w0, up, down, after, before, gate = p[0], p[1:3], p[3:5], p[5:7], p[7:9], p[9:11]
    h, u = x, normed(x, w0)
    for i in range(2):
        a, b = (u @ up[i].t()).chunk(2, -1)
        y = (a * torch.sigmoid(a) * b) @ down[i].t()
        h = h + gate[i] * normed(y, after[i])
        u = normed(h, before[i])
    return u, p


def _linear(x, w):
    return x @ w.to(x.dtype).t()


def test_blocks_against_float64():
    """fp32 throughout, library products for the linear layers: the layers' own
    errors, through two blocks, stay within 2^-12 of each tensor's norm (a few
    hundred roundings of 2^-24 a layer, 10 layers, amplified at most 4-fold by
    the weights' norms of a block)."""
    net = Blocks(96, 160)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, du = normal(gen, 50, 96), normal(gen, 50, 96)
    xg = x.clone().requires_grad_()
    u = net.forward(xg, "same", _linear)
    got = torch.autograd.grad(u, [xg] + net.parameters(), du)
    xd = x.cpu().double().requires_grad_()
    want_u, p = _plain_forward(net, xd, _linear)
    want = torch.autograd.grad(want_u, [xd] + p, du.cpu().double())
    for g, w in zip((u, *got), (want_u, *want)):
        assert (g.cpu().double() - w).norm() <= 2.0 ** -12 * w.norm()


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_blocks_with_8_bit_checkpoints(dtype):
    """The same outputs; gradients within the rounding of what was kept: each kept
    value is off by 2^-4 of itself at most, at random, and five layers' worth of such
    errors (relative 2^-4 / sqrt 3 each, in part of a gradient's factors)
    stay below a quarter of a gradient's norm.  Library products between the
    layers: those of mx4 round the gradients to 4 bits anew, which would
    be compared here instead."""
    net = Blocks(128, 256)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, du = normal(gen, 64, 128, dtype=dtype), normal(gen, 64, 128, dtype=dtype)
    out = {}
    for keep in ("same", "mx8"):
        xg = x.clone().requires_grad_()
        u = net.forward(xg, keep, _linear)
        out[keep] = (u.detach(), *torch.autograd.grad(u, [xg] + net.parameters(), du))
    assert torch.equal(out["same"][0], out["mx8"][0])
    for a, b in zip(out["same"][1:], out["mx8"][1:]):
        assert torch.isfinite(b).all() and (a - b).float().norm() <= 0.25 * a.float().norm()


def test_8_bit_checkpoints_hold_half_the_memory():
    """What a layer keeps: 1.03 bytes an element of its inputs and 8 bytes a row and norm.  The
    inputs themselves are freed, but for a residual stream that is the caller's."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows, cols = 512, 1024
    kept = rows * cols * 33 // 32
    r = normal(gen, rows, cols, dtype=BF16).requires_grad_()
    n = L.Norm("rms", torch.ones(cols, device="cuda", requires_grad=True))

    def held(make, f):
        t = make()
        gc.collect()
        base = torch.cuda.memory_allocated()
        out = f(t)
        size = t.numel() * t.element_size()
        del t
        gc.collect()
        outs = [o for o in (out if isinstance(out, tuple) else (out,)) if o is not None]
        return torch.cuda.memory_allocated() - base + size - sum(o.numel() * o.element_size() for o in outs)

    def one():
        return r * 1.0

    def two():
        return torch.cat((r, r), 1)
    slack = 4096
    assert held(one, lambda t: L.activation(t, keep="mx8")) <= kept + slack
    assert held(two, lambda t: L.gated(t, keep="mx8")) <= 2 * kept + slack
    assert held(one, lambda t: L.norm(t, n, keep="mx8")) <= kept + 8 * rows + slack
    assert held(one, lambda t: L.join(r, t, n, None, 1.0, n, "mx8")) <= 2 * kept + 16 * rows + slack
    assert held(one, lambda t: L.activation(t)) >= 2 * rows * cols


def test_serving_single_rows():
    """One row at a time through the same layers, from MX4 weights, as all rows at once."""
    net = Blocks(128, 256)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = normal(gen, 9, 128, dtype=BF16)
    weights = {id(w): MX.quantize(w.detach()) for w in net.up + net.down}
    with torch.no_grad():
        def linear(t, w):
            return MX.linear(t, weights[id(w)])
        whole = net.forward(x, "same", linear)
        rows = torch.cat([net.forward(row[None], "same", linear) for row in x])
    assert torch.equal(whole, rows)


def test_a_captured_training_step_replays():
    net = Blocks(64, 96)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, du = normal(gen, 40, 64, dtype=BF16), normal(gen, 40, 64, dtype=BF16)

    def step(t):
        t = t.detach().requires_grad_()
        u = net.forward(t, "mx8")
        return [u.detach(), *torch.autograd.grad(u, [t] + net.parameters(), du)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static)
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(100 + seed)
        static.copy_(normal(gen, 40, 64, dtype=BF16))
        want = step(static)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_a_captured_backward_pass_beside_an_eager_graph_is_refused():
    """The leaf's gradient would go to a node on the eager graph's stream; freed, the capture works."""
    x = torch.randn(40, 64, device="cuda", requires_grad=True)
    n = L.Norm("rms", torch.ones(64, device="cuda", requires_grad=True))
    for f in (lambda: L.activation(x, keep="mx8"), lambda: L.norm(x, n, keep="mx8")):
        eager = f()
        dy = torch.ones_like(eager)
        torch.cuda.synchronize()
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            y = f()
            with pytest.raises(RuntimeError, match="before the capture"):
                torch.autograd.grad(y, x, dy)
        want = torch.autograd.grad(eager, x, dy)[0]
        del eager, y
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = torch.autograd.grad(f(), x, dy)[0]
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_two_captured_graphs_in_turn():
    """Each has its own workspace: replays of one leave the other's results alone."""
    net = Blocks(64, 96)
    gen = torch.Generator(device="cuda").manual_seed(9)
    xs = [normal(gen, rows, 64, dtype=BF16) for rows in (40, 33)]
    dus = [normal(gen, rows, 64, dtype=BF16) for rows in (40, 33)]

    def step(t, du):
        t = t.detach().requires_grad_()
        return torch.autograd.grad(net.forward(t, "mx8"), [t] + net.parameters(), du)
    want = [step(x, du) for x, du in zip(xs, dus)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, du in zip(xs, dus):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(x, du))
    for turn in range(3):
        for g in graphs:
            g.replay()
        step(xs[turn % 2], dus[turn % 2])
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_two_threads_at_once():
    net = Blocks(64, 96)
    gen = torch.Generator(device="cuda").manual_seed(10)
    xs = [normal(gen, 40 + 7 * i, 64, dtype=BF16) for i in range(4)]

    def step(t):
        t = t.detach().requires_grad_()
        u = net.forward(t, "mx8")
        return torch.autograd.grad(u, [t] + net.parameters(), torch.ones_like(u))
    want = [step(x) for x in xs]
    torch.cuda.synchronize()

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got = step(xs[i])
            torch.cuda.current_stream().synchronize()
        return all(torch.equal(a, b) for a, b in zip(got, want[i]))
    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(run, range(4)))


def test_on_a_side_stream():
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = normal(gen, 300, 256, dtype=BF16)
    n = L.Norm("layer", torch.ones(256, device="cuda", requires_grad=True))

    def step(t):
        t = t.detach().requires_grad_()
        h, u = L.join(t, L.gated(torch.cat((t, t), 1), keep="mx8"), n, None, 1.0, n, "mx8")
        return torch.autograd.grad((h, u), (t, n.weight), (torch.ones_like(h), torch.ones_like(u)))
    want = step(x)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step(x))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_recomputed_in_a_checkpoint_and_offloaded():
    from torch.utils.checkpoint import checkpoint
    net = Blocks(64, 96)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, du = normal(gen, 40, 64).requires_grad_(), normal(gen, 40, 64)
    leaves = [x] + net.parameters()
    want = torch.autograd.grad(net.forward(x, "mx8"), leaves, du)
    got = torch.autograd.grad(checkpoint(lambda t: net.forward(t, "mx8"), x, use_reentrant=False), leaves, du)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.cpu(), lambda t: t.cuda()):
        u = net.forward(x, "mx8")
    got = torch.autograd.grad(u, leaves, du)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_retained_graphs_and_freed_ones():
    n = L.Norm("rms", torch.ones(64, device="cuda", requires_grad=True))
    x = torch.randn(30, 64, device="cuda", requires_grad=True)
    for f in (lambda: L.activation(x, keep="mx8"), lambda: L.gated(x), lambda: L.norm(x, n),
              lambda: L.join(x, x, n, None, 1.0, n)[1]):
        y = f().square().sum()
        a = torch.autograd.grad(y, x, retain_graph=True)[0]
        assert torch.equal(a, torch.autograd.grad(y, x)[0])
        with pytest.raises(RuntimeError, match="second time"):
            torch.autograd.grad(y, x)


def test_changed_inputs_are_noticed():
    """Kept as they are, inputs may not change before backward; their 8-bit copies do not see it."""
    for keep in ("same", "mx8"):
        leaf = torch.randn(8, 64, device="cuda", requires_grad=True)
        x = leaf * 1.0
        y = L.activation(x, keep=keep)
        x.add_(1.0)
        if keep == "same":
            with pytest.raises(RuntimeError, match="modified by an inplace"):
                torch.autograd.grad(y.sum(), leaf)
        else:
            got = torch.autograd.grad(y.sum(), leaf)[0]
            want = O.act(O.mx8_values(leaf.detach().cpu()), "silu")[1]
            assert (got.cpu() - want).abs().max() < 1e-5


def test_gradients_of_gradients_and_tangents_are_refused():
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    n = L.Norm()
    for f in (L.activation, L.gated, lambda t: L.norm(t, n), lambda t: L.join(t, t, n)[0]):
        g, = torch.autograd.grad(f(x).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.sum(), x)
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(x.detach(), torch.ones_like(x))
            with pytest.raises(NotImplementedError):
                f(dual)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_inside_saved_tensors(dtype):
    """Layers that keep their inputs take them rounded, as with keep="mx8"; row statistics are left alone."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, r = normal(gen, 300, 256, dtype=dtype).requires_grad_(), normal(gen, 300, 256, dtype=dtype).requires_grad_()
    dy = normal(gen, 300, 256, dtype=dtype)
    n = L.Norm("layer", (1 + normal(gen, 256, std=0.1)).requires_grad_())

    def step(keep):
        y = L.activation(x * 1.0, act="gelu", keep=keep)
        h, u = L.join(r * 1.0, y, n, None, 1.0, n, keep)
        return L.norm(h, n, keep=keep) + u
    want = torch.autograd.grad(step("mx8"), (x, r, n.weight), dy)
    with M8.saved_tensors(min_elements=512, dtypes=(dtype,)):
        out = step("same")
    got = torch.autograd.grad(out, (x, r, n.weight), dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
