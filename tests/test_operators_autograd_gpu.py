"""What autograd may expect of the MX4 layers: gradients that a call cannot form
are refused, and what backward needs is kept the way autograd frees and moves it."""
import gc

import pytest
import torch
from torch.autograd import forward_ad

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx4 as MX

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _pair(rows=40, n=96, k=160):
    gen = torch.Generator(device="cuda").manual_seed(3)
    return torch.randn(rows, k, generator=gen, device="cuda"), torch.randn(n, k, generator=gen, device="cuda")


@pytest.mark.parametrize("rows", [1, 40])
def test_linear_refuses_an_input_that_requires_grad(rows):
    x, w = _pair(rows)
    q = MX.quantize(w)
    want = MX.linear(x, q)
    x.requires_grad_()
    for bad in (x, x * 1.0, x.view(rows, 1, -1)):
        with pytest.raises(ValueError, match="gradient"):
            MX.linear(bad, q)
    with torch.no_grad():
        assert torch.equal(MX.linear(x, q), want)
    assert torch.equal(MX.linear(x.detach(), q), want)


def test_outputs_that_require_grad_are_refused():
    x, w = _pair()
    q, xq = MX.quantize(w), MX.quantize(x)
    out = torch.zeros(40, 96, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        MX.linear(x, q, out=out)
    with pytest.raises(ValueError, match="gradient"):
        MX.product(xq, q, out=out)
    with torch.no_grad():
        assert torch.equal(MX.linear(x, q, out=out), MX.product(xq, q, dtype=torch.float32))


def test_forward_mode_tangents_are_refused():
    x, w = _pair()
    q = MX.quantize(w)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        dual_w = forward_ad.make_dual(w, torch.ones_like(w))
        with pytest.raises(ValueError, match="tangent"):
            MX.linear(dual, q)
        for args in ((dual, w), (x, dual_w)):
            with pytest.raises(NotImplementedError, match="jvp"):
                MX.train_linear(*args)
            with torch.no_grad(), pytest.raises(NotImplementedError, match="jvp"):
                MX.train_linear(*args)
        assert torch.equal(MX.train_linear(x, w), MX.train_linear(x, w))
        MX.linear(x, q)


def test_backward_frees_what_it_used():
    x, w = _pair()
    x.requires_grad_(), w.requires_grad_()
    before = torch.cuda.memory_allocated()
    y = MX.train_linear(x, w)
    held = torch.cuda.memory_allocated() - before
    loss = y.sum()
    node = y.grad_fn
    del y
    loss.backward()
    x.grad = w.grad = None
    gc.collect()
    # the loss and its graph are still there, the quantised copies are not
    assert loss.grad_fn is not None and node is not None
    assert torch.cuda.memory_allocated() - before <= 1024, (held, torch.cuda.memory_allocated() - before)
    with pytest.raises(RuntimeError, match="second time"):
        loss.backward()


def test_a_retained_graph_gives_the_same_gradients_again():
    x, w = _pair()
    x.requires_grad_(), w.requires_grad_()
    y = MX.train_linear(x, w).square().sum()
    a = torch.autograd.grad(y, (x, w), retain_graph=True)
    b = torch.autograd.grad(y, (x, w))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_saved_tensor_hooks_see_what_backward_needs():
    """Offloading: every saved tensor goes to the host and comes back elsewhere."""
    x, w = _pair()
    x.requires_grad_(), w.requires_grad_()
    want = torch.autograd.grad(MX.train_linear(x, w).square().sum(), (x, w))
    moved = []

    def pack(t):
        moved.append(t.numel() * t.element_size())
        return t.cpu()
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.cuda()):
        y = MX.train_linear(x, w)
    assert sum(moved) >= (160 * 128 + 160 * 128) * 17 // 32        # x^T and w^T in MX4
    got = torch.autograd.grad(y.square().sum(), (x, w))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_recomputed_in_a_checkpoint():
    from torch.utils.checkpoint import checkpoint
    x, w = _pair()
    x.requires_grad_(), w.requires_grad_()
    f = lambda a, b: MX.train_linear(a, b).relu()  # noqa: E731
    want = torch.autograd.grad(f(x, w).square().sum(), (x, w))
    gc.collect()
    before = torch.cuda.memory_allocated()
    y = checkpoint(f, x, w, use_reentrant=False)
    assert torch.cuda.memory_allocated() - before <= 40 * 96 * 4 + 1024   # the output alone
    got = torch.autograd.grad(y.square().sum(), (x, w))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
