"""Joins whose branch has infinities and NaN: gradients that do not depend on the
branch stay finite."""
import itertools
import math

import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from layers_helpers import check, normal

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (F32, BF16), (BF16, BF16)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


@pytest.mark.parametrize("gate", [None, "channel", "sequence", "row", "token"])
@pytest.mark.parametrize("keep", ["same", "mx8"])
@pytest.mark.parametrize("types", TYPES, ids=["f32", "mixed", "bf16"])
@pytest.mark.parametrize("cols", [40, 2050, 9000])
def test_gradient_of_a_branch_that_is_not_finite(gate, keep, types, cols):
    """Without a norm after it the branch's gradient is gate dh, whatever the branch is: one
    product (and the gradient's rounding), also beside neighbours in the same group of 32."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    shape = (2, 3, cols)
    size = {"channel": (cols,), "sequence": (2, 1, cols), "row": shape, "token": (2, 3, 1)}.get(gate)
    for before, biased in itertools.product((None, "rms", "layer"), (False, True)):
        r = normal(gen, *shape, dtype=types[0]).requires_grad_()
        y = normal(gen, *shape, dtype=types[1])
        y[0, 0, 1], y[0, 1, 7], y[1, 0, cols - 1], y[1, 2, 33] = math.inf, math.nan, -math.inf, math.inf
        y.requires_grad_()
        g = None if gate is None else (normal(gen, *size, std=0.5) + 0.5).requires_grad_()
        # a bias of the next norm takes the kernels with biases; its output has no gradient here
        n = before and L.Norm(before, bias=torch.zeros(cols, device="cuda") if biased else None)
        h, _ = L.join(r, y, gate=g, scale=0.5, before=n, keep=keep)
        dh = normal(gen, *shape, dtype=types[0])
        dr, dy = torch.autograd.grad(h, (r, y), dh)
        want = dh.double() if g is None else dh.double() * g.detach().double()
        check(dy, want, want.abs(), 2, f"{before} {biased} branch")
        check(dr, 0.5 * dh.double(), dh.double().abs(), 1, "residual")
        bad = ~torch.isfinite(y)
        assert torch.isfinite(h[~bad]).all() and not torch.isfinite(h[bad]).any()
