"""The layers under torch's transforms: run between the graphs of torch.compile, refused by torch.func and in traces."""
import pytest
import torch
from torch.fx.experimental.proxy_tensor import make_fx

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from inverse_root_preconditioning_amd import mx8 as M8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _forms(w):
    n = L.Norm("rms", w)
    return {"activation": lambda t: L.activation(t, keep="mx8"), "gated": lambda t: L.gated(t),
            "norm": lambda t: L.norm(t, n), "join": lambda t: L.join(t, t * 2, n, None, 1.0, n, "mx8")[1]}


def test_compiled_functions_call_them():
    """Without a code generator: the graphs around the calls run as they are."""
    x = torch.randn(6, 64, device="cuda", requires_grad=True)
    w = torch.randn(64, device="cuda", requires_grad=True)
    for name, f in _forms(w).items():
        def whole(t):
            return f(t * 2) + 1
        fast = torch.compile(whole, backend="eager")
        got, want = fast(x), whole(x)
        assert torch.equal(got, want), name
        for a, b in zip(*(torch.autograd.grad(y.sum(), (x, w), allow_unused=True) for y in (got, want))):
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b)), name


def test_function_transforms_are_refused():
    x, w = torch.randn(3, 6, 64, device="cuda"), torch.randn(64, device="cuda")
    for name, f in _forms(w).items():
        for transform in (lambda: torch.func.grad(lambda t: f(t).sum())(x), lambda: torch.vmap(f)(x),
                          lambda: torch.func.jvp(f, (x,), (x,)), lambda: torch.func.vjp(f, x)):
            with pytest.raises(RuntimeError):
                transform()
    with pytest.raises(RuntimeError):
        torch.vmap(lambda v: L.norm(x, L.Norm("rms", v)))(w.expand(3, 64).contiguous())


def test_batched_gradients_are_refused():
    x, w = torch.randn(6, 64, device="cuda", requires_grad=True), torch.randn(64, device="cuda")
    for f in _forms(w).values():
        y = f(x)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(y, x, torch.ones(2, *y.shape, device="cuda"), is_grads_batched=True)


def test_traces_are_refused():
    x, w = torch.randn(6, 64, device="cuda"), torch.randn(64, device="cuda")
    forms = {**_forms(w), "mx8": lambda t: M8.dequantize(M8.quantize(t))}
    for f in forms.values():
        with pytest.raises(NotImplementedError, match="trace"):
            torch.jit.trace(f, x, check_trace=False)
        with pytest.raises(NotImplementedError, match="trace"):
            make_fx(f)(x)
        f(x)


def test_a_trace_inside_saved_tensors():
    """Of torch's own operations: what they save stays as it is."""
    x = torch.randn(64, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)

    def f(t):
        return torch.sin(t * 1)
    with M8.saved_tensors(min_elements=64):
        traced = torch.jit.trace(f, x, check_trace=False)
    assert torch.equal(traced(x), f(x))
