"""Tensors that only stand for others (wrapper subclasses, as sharded or quantised ones are) have no memory
for a kernel to read: they are refused, whichever argument they are."""
import pytest
import torch
from torch.utils._pytree import tree_map

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from inverse_root_preconditioning_amd import mx8 as M8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


class Wrapper(torch.Tensor):
    @staticmethod
    def __new__(cls, inner):
        return torch.Tensor._make_wrapper_subclass(cls, inner.size(), strides=inner.stride(), dtype=inner.dtype,
                                                   device=inner.device, requires_grad=False)

    def __init__(self, inner):
        self.inner = inner

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        args, kwargs = tree_map(lambda t: t.inner if isinstance(t, cls) else t, (args, kwargs or {}))
        return func(*args, **kwargs)


@pytest.mark.parametrize("which", ["x", "branch", "weight", "bias", "gate", "token"])
@pytest.mark.parametrize("grad", [False, True])
def test_wrappers_are_refused(which, grad):
    x, y = torch.randn(3, 64, device="cuda", requires_grad=grad), torch.randn(3, 64, device="cuda")
    w, b = torch.randn(64, device="cuda"), torch.randn(64, device="cuda")
    gate, token = torch.randn(64, device="cuda"), torch.randn(3, 1, device="cuda")
    one = {"x": x, "branch": y, "weight": w, "bias": b, "gate": gate, "token": token}
    one[which] = Wrapper(one[which].detach())
    g = one["token"] if which == "token" else one["gate"]
    n = L.Norm("rms", one["weight"], one["bias"])
    with pytest.raises((ValueError, RuntimeError)):
        L.join(one["x"], one["branch"], n, g)
    if which in ("x", "weight", "bias"):
        with pytest.raises((ValueError, RuntimeError)):
            L.norm(one["x"], n)
    if which in ("x", "branch"):
        with pytest.raises((ValueError, RuntimeError)):
            L.gated(one["x"], one["branch"])
    if which == "x":
        with pytest.raises((ValueError, RuntimeError)):
            M8.quantize(one["x"])
