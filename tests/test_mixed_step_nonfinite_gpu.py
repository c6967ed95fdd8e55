"""A gradient that is not finite leaves the example's whole network unchanged."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("which", [0, 3])
def test_example_survives_a_gradient_that_is_not_finite(which, monkeypatch):
    """The third and the sixth step (where roots are made anew) get a NaN in a
    matrix's or a vector's gradient; the loss still falls."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import mixed_step
    real, calls = torch.autograd.grad, []

    def grad(*args, **kw):
        out = list(real(*args, **kw))
        calls.append(1)
        if len(calls) in (3, 6):
            out[which] = out[which].clone()
            out[which].view(-1)[5] = float("nan")
        return out
    monkeypatch.setattr(torch.autograd, "grad", grad)
    losses, off = mixed_step.train(steps=40, log=lambda s: print(s, flush=True))
    assert all(math.isfinite(v) for v in losses)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5]) and off < 1e-2
