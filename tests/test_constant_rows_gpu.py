"""Layer norms of rows of one value: x - mean is 0, and so is what is formed from it."""
import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L
from layers_helpers import normal

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (F32, BF16), (BF16, BF16)]
# Sums over a row are exact: 96 and 30720 are 3 * 2^5 and 15 * 2^11, 3.5 is 7 / 2, and 15 * 16384 < 2^24; so is
# the mean, the quotient of such a sum by the columns.  All have at most 4 significant bits, as MX8 codes hold.
VALUES = (96.0, 30720.0, -3.5, 0.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


@pytest.mark.parametrize("keep", ["same", "mx8"])
@pytest.mark.parametrize("types", TYPES, ids=["f32", "mixed", "bf16"])
@pytest.mark.parametrize("cols", [1, 3, 64, 777, 1000, 2048, 5000, 8192, 16384])
def test_norm_is_its_bias(cols, types, keep):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.tensor(VALUES, device="cuda").to(types[0])[:, None].expand(-1, cols).contiguous().requires_grad_()
    n = L.Norm("layer", normal(gen, cols).requires_grad_(), normal(gen, cols).requires_grad_(), 1e-6)
    u = L.norm(x, n, dtype=types[1], keep=keep)
    assert torch.equal(u, n.bias.detach().to(types[1]).expand_as(u))
    dx, dw = torch.autograd.grad(u, (x, n.weight), normal(gen, len(VALUES), cols, dtype=types[1]))
    assert torch.equal(dw, torch.zeros_like(dw))
    assert torch.isfinite(dx).all()


def test_norm_of_a_value_with_more_bits():
    """101 and 30080 (235 * 2^7) in rows of a power of two."""
    x = torch.tensor([101.0, 30080.0], device="cuda")[:, None].expand(-1, 512).contiguous()
    for eps in (1e-6, 1e-5):
        assert not L.norm(x, L.Norm("layer", eps=eps)).any()


@pytest.mark.parametrize("keep", ["same", "mx8"])
@pytest.mark.parametrize("types", TYPES, ids=["f32", "mixed", "bf16"])
@pytest.mark.parametrize("cols", [1, 100, 2048, 5000, 9000, 16384])
def test_join_of_constant_rows(cols, types, keep):
    """z = 0 after the first norm, h = r, a constant row again, and u the second norm's bias."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    v = torch.tensor(VALUES, device="cuda")[:, None].expand(-1, cols)
    r, y = v.to(types[0]).contiguous().requires_grad_(), v.flip(0).to(types[1]).contiguous().requires_grad_()
    w1, w2, b2 = (normal(gen, cols).requires_grad_() for _ in range(3))
    h, u = L.join(r, y, after=L.Norm("layer", w1), before=L.Norm("layer", w2, b2), keep=keep)
    assert torch.equal(h, r) and torch.equal(u, b2.detach().to(types[1]).expand_as(u))
    dh, du = normal(gen, *h.shape, dtype=types[0]), normal(gen, *u.shape, dtype=types[1])
    dw1, dw2 = torch.autograd.grad((h, u), (w1, w2), (dh, du))
    assert torch.equal(dw1, torch.zeros_like(dw1)) and torch.equal(dw2, torch.zeros_like(dw2))
