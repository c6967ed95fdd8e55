"""MX4 linear layers whose output lies beside their input in one buffer, or over it."""
import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx4 as MX

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


@pytest.mark.parametrize("rows", [1, 3, 16, 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_input_and_output_in_one_buffer(rows, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    w = MX.quantize(torch.randn(96, 160, generator=gen, device="cuda"))
    x = torch.randn(rows, 160, generator=gen, device="cuda").to(dtype)
    want = MX.linear(x, w)
    for first in (0, 96, 101):                       # the output's columns after or before the input's
        buf = torch.zeros(rows, 300, dtype=dtype, device="cuda")
        a, b = (buf[:, :160], buf[:, 160:256]) if first == 0 else (buf[:, first:first + 160], buf[:, :96])
        a.copy_(x)
        assert torch.equal(MX.linear(a, w, out=b), want) and torch.equal(a, x)
        used = torch.zeros(300, dtype=torch.bool)
        used[slice(0, 256) if first == 0 else slice(first, first + 160)] = True
        used[:96] = True
        assert bool((buf[:, ~used.cuda()] == 0).all())
    whole = torch.zeros(2 * rows, 160, dtype=dtype, device="cuda")    # one after the other
    whole[:rows] = x
    assert torch.equal(MX.linear(whole[:rows], w, out=whole[rows:, :96]), want)


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_an_output_over_the_input_is_refused(rows):
    w = MX.quantize(torch.randn(64, 64, device="cuda"))
    x = torch.randn(rows, 64, device="cuda")
    was = x.clone()
    with pytest.raises(capi.ShampooError):
        MX.linear(x, w, out=x)
    buf = torch.zeros(rows, 127, device="cuda")
    with pytest.raises(capi.ShampooError):
        MX.linear(buf[:, :64], w, out=buf[:, 63:])
    torch.cuda.synchronize()
    assert torch.equal(x, was) and bool((buf == 0).all())
