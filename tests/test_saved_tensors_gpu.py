"""What mx8.saved_tensors rounds: activations, and no weights."""
import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx8 as M8
from layers_helpers import normal

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
F = torch.nn.functional


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _input_gradient(h, f, dy, rounded):
    """The gradient of h's leaf through f, inside a context that keeps what it may in 8 bits."""
    leaf = h.detach().clone().requires_grad_()
    t = leaf * 1
    if rounded:
        with M8.saved_tensors(min_elements=64):
            y = f(t)
    else:
        y = f(t)
    return torch.autograd.grad(y, leaf, dy)[0]


def _autocast(t, w):
    with torch.autocast("cuda", dtype=BF16):
        return F.linear(t, w)


@pytest.mark.parametrize("form", ["frozen", "frozen tensor", "cast", "frozen cast", "autocast", "frozen autocast",
                                  "cast of a view", "cast of a part", "cast of a split part", "cast of parts unbound"])
def test_weights_are_left_alone(form):
    """A linear layer's input gradient is dy W: the same bits with and without the context, whether the
    weight is trained or not, and where it is a cast of an fp32 one."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = normal(gen, 40, 96, dtype=BF16)
    dy = normal(gen, 40, 64, dtype=BF16)
    w32 = torch.nn.Parameter(normal(gen, 64, 96), requires_grad="frozen" not in form)
    two, three = normal(gen, 74, 96).requires_grad_(), normal(gen, 2, 1, 64, 96).requires_grad_()
    w16 = torch.nn.Parameter(w32.detach().to(BF16), requires_grad=False)
    f = {"frozen": lambda t: F.linear(t, w16), "frozen tensor": lambda t: t @ w16.data.t(),
         "cast": lambda t: F.linear(t, w32.to(BF16)), "frozen cast": lambda t: F.linear(t, w32.to(BF16)),
         "autocast": lambda t: _autocast(t, w32), "frozen autocast": lambda t: _autocast(t, w32),
         "cast of a view": lambda t: t @ w32.view(64, 96).t().to(BF16),
         "cast of a part": lambda t: F.linear(t, two[:64].to(BF16)),
         "cast of a split part": lambda t: F.linear(t, two.split([64, 10])[0].to(BF16)),
         "cast of parts unbound": lambda t: F.linear(t, three.unbind()[1].squeeze(0).to(BF16))}[form]
    assert torch.equal(_input_gradient(h, f, dy, True), _input_gradient(h, f, dy, False))


def test_frozen_weights_take_no_memory():
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.nn.Parameter(normal(gen, 512, 512, dtype=BF16), requires_grad=False)
    t = normal(gen, 8, 512, dtype=BF16).requires_grad_() * 1
    F.linear(t.detach(), w)                      # the library's own workspace
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    with M8.saved_tensors():
        y = F.linear(t, w)
    assert torch.cuda.memory_allocated() - before <= y.numel() * 2 + 1024


def test_masks_are_left_alone():
    """A dropout keeps 0 and 1 / (1 - p), which 4 bits of a value do not hold."""
    h = torch.ones(64, 96, device="cuda", dtype=BF16)
    mask = (torch.rand(64, 96, device="cuda") < 0.7).to(BF16) * 1.4296875
    dy = torch.ones_like(h)
    assert torch.equal(_input_gradient(h, lambda t: t * mask, dy, True), mask)


def test_a_function_with_an_attribute_of_its_own():
    """What a caller's function calls its values does not make its output a leaf."""
    class Twice(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            ctx.variable = 2
            return t * 2

        @staticmethod
        def backward(ctx, dy):
            return dy * 2
    h = torch.randn(40, 96, device="cuda", dtype=BF16)
    leaf = h.clone().requires_grad_()
    with M8.saved_tensors(min_elements=64):
        y = torch.sin(Twice.apply(leaf))
    h8 = M8.dequantize(M8.quantize(h * 2), BF16)
    assert torch.equal(torch.autograd.grad(y, leaf, torch.ones_like(y))[0], torch.cos(h8) * 2)


def test_activations_are_still_rounded():
    gen = torch.Generator(device="cuda").manual_seed(3)
    h = normal(gen, 40, 96, dtype=BF16)
    w = normal(gen, 64, 96, dtype=BF16).requires_grad_()
    dy = normal(gen, 40, 64, dtype=BF16)
    t = h.clone().requires_grad_() * 1
    with M8.saved_tensors(min_elements=64):
        y = F.linear(t, w)
    dw, = torch.autograd.grad(y, w, dy)
    h8 = M8.dequantize(M8.quantize(h), BF16)
    u = h8.clone().requires_grad_()
    want, = torch.autograd.grad(F.linear(u, w), w, dy)
    assert torch.equal(dw, want)
