"""Memory of a join's backward pass with a gate of the matrix's own size."""
import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from layers_helpers import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


@pytest.mark.parametrize("bias", [False, True])
def test_no_workspace_for_gradients_that_nobody_wants(bias):
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows, cols = 1 << 14, 256
    r, y = normal(gen, rows, cols).requires_grad_(), normal(gen, rows, cols).requires_grad_()
    gate, w1, w2 = normal(gen, rows, cols), normal(gen, cols), normal(gen, cols)
    b1 = normal(gen, cols) if bias else None
    dh, du = normal(gen, rows, cols), normal(gen, rows, cols)
    got = {}
    for wanted in (False, True):
        gate.requires_grad_(wanted), w1.requires_grad_(wanted)
        h, u = L.join(r, y, L.Norm("rms", w1, b1), gate, 1.0, L.Norm("layer", w2))
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        got[wanted] = torch.autograd.grad((h, u), (r, y) + ((gate, w1) if wanted else ()), (dh, du))
        held = torch.cuda.max_memory_allocated() - before
        matrix = rows * cols * 4
        if wanted:
            assert held <= (3 + 1 + bias) * matrix + (1 << 22)
        else:
            assert held <= 2 * matrix + (1 << 22)
    assert torch.equal(got[False][0], got[True][0]) and torch.equal(got[False][1], got[True][1])
