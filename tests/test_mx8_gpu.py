"""MX8 rows against the float64 oracle: codes and scales equal, values exact."""
import math

import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx8 as M8
from oracle import layers_oracle as O
from layers_helpers import strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _equal(x, q):
    codes, scales = O.mx8_codes(x.cpu())
    assert q.shape == tuple(x.shape) and q.codes.shape == codes.shape and q.scales.shape == scales.shape
    assert torch.equal(q.scales.cpu().long(), scales)
    got = q.codes.cpu().long()
    assert torch.equal(got, codes), ((got != codes).sum(), x.cpu().flatten()[(got[:, :x.shape[1]] != codes[:, :x.shape[1]]).flatten()][:4])
    want = O.mx8_decode(codes, scales, x.shape[1])
    for dtype in (torch.float32, torch.bfloat16):
        v = M8.dequantize(q, dtype).cpu()
        assert v.dtype == dtype and v.shape == x.shape
        assert torch.equal(torch.nan_to_num(v.double(), nan=7.0), torch.nan_to_num(want.to(dtype).double(), nan=7.0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3), (2, 7), (1, 31), (3, 32), (5, 33), (7, 100), (66, 257), (64, 1001),
                                       (130, 2048), (17, 4099)])
@pytest.mark.parametrize("layout", ["plain", "padded"])
def test_codes_scales_and_values(rows, cols, dtype, layout):
    gen = torch.Generator(device="cuda").manual_seed(rows * 10007 + cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(4 * torch.randn(rows, cols, generator=gen, device="cuda"))   # many binades in a group
    x = strided(x.to(dtype), layout)
    _equal(x, M8.quantize(x))


@pytest.mark.parametrize("top", [1.0, 1.9375, 2.0 ** -126, 2.0 ** -118, 2.0 ** 127, 3.0e38])
def test_every_bf16_value_beside_a_largest_one(top):
    """All bf16 numbers below the largest of their group, subnormals and ties among them."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x) & (x.double().abs() <= top)]
    x = torch.nn.functional.pad(x, (0, -x.numel() % 31)).view(-1, 31)
    x = torch.cat((x, torch.full((x.shape[0], 1), top, dtype=torch.bfloat16)), 1).cuda()
    _equal(x, M8.quantize(x))
    _equal(x.float(), M8.quantize(x.float()))


def test_fp32_neighbours_of_every_border():
    """Both fp32 neighbours of each value halfway between two codes, and the value."""
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    near = table[torch.isfinite(table) & (table.abs() <= 256)].unique()
    tie = ((near[1:] + near[:-1]) / 2).float()
    tie = tie[tie.abs() < 256]
    x = torch.cat((tie, torch.nextafter(tie, torch.tensor(math.inf)), torch.nextafter(tie, torch.tensor(-math.inf))))
    x = torch.nn.functional.pad(x, (0, -x.numel() % 31)).view(-1, 31)
    x = torch.cat((x, torch.full((x.shape[0], 1), 255.0)), 1)
    for e in (0, -100, 100, -125):
        y = torch.ldexp(x, torch.tensor(e)).cuda()
        _equal(y, M8.quantize(y))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_special_groups(dtype):
    x = torch.ones(8, 70, device="cuda", dtype=dtype)
    x[0, 33] = math.nan
    x[1, 64] = math.inf
    x[2, 69] = -math.inf
    x[3] = 0.0
    x[4] = -0.0
    x[5] = torch.finfo(dtype).max
    x[6] = torch.finfo(dtype).tiny
    x[7] = 1e-40
    q = M8.quantize(x)
    _equal(x, q)
    v = M8.dequantize(q)
    assert torch.isnan(v[0, 32:64]).all() and not torch.isnan(v[0, :32]).any()
    assert torch.isnan(v[1, 64:]).all() and torch.isnan(v[2, 64:]).all() and not torch.isnan(v[2, :64]).any()


def test_empty_and_repeated():
    for shape in ((0, 5), (5, 0)):
        x = torch.zeros(shape, device="cuda")
        assert M8.dequantize(M8.quantize(x)).shape == shape
    x = torch.randn(300, 700, device="cuda")
    a, b = M8.quantize(x), M8.quantize(x)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    again = M8.MX8Matrix(a.codes.clone(), a.scales.clone(), 300, 700)
    assert torch.equal(M8.dequantize(again), M8.dequantize(a))


def test_on_another_stream():
    s = torch.cuda.Stream()
    x = torch.randn(100, 300, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    v = M8.dequantize(M8.quantize(x, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(v, M8.dequantize(M8.quantize(x)))


def test_rows_beyond_32_bit_offsets():
    """A matrix of 2^32 + 2^23 bytes and more: the last rows are those of a small one."""
    rows, cols = (1 << 19) + 1024, 4096
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    tail = torch.randn(5, cols, device="cuda").to(torch.bfloat16)
    x[-5:] = tail
    q = M8.quantize(x)
    assert torch.equal(q.codes[-5:], M8.quantize(tail).codes)
    v = M8.dequantize(q, torch.bfloat16)
    assert torch.equal(v[-5:], M8.dequantize(M8.quantize(tail), torch.bfloat16)) and not v[:100].any()


def test_refusals():
    x = torch.randn(4, 64, device="cuda")
    for bad in (x.half(), x.cpu(), x[0], x.t()):
        with pytest.raises(ValueError):
            M8.quantize(bad)
    q = M8.quantize(x)
    with pytest.raises(ValueError):
        M8.dequantize(q, torch.float16)
    with pytest.raises(ValueError):
        M8.MX8Matrix(q.codes, q.scales, 4, 65)
    with pytest.raises(ValueError):
        M8.MX8Matrix(q.codes.cpu(), q.scales, 4, 64)


def test_saved_tensors_are_kept_in_8_bits():
    """sin(x) saves x: its gradient is dy cos of the rounded x.  Parameters and views of them stay as they are."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(96, 200, generator=gen, device="cuda")
    w = torch.randn(300, 200, generator=gen, device="cuda", requires_grad=True)
    xg = x.clone().requires_grad_()
    with M8.saved_tensors(min_elements=64, dtypes=(torch.float32,)):
        h = xg * 1.0
        before = torch.cuda.memory_allocated()
        y = torch.sin(h)
        held = torch.cuda.memory_allocated() - before - y.numel() * 4
        z = y @ w.t()
    assert held <= 96 * 224 * 34 // 32 + 512
    dz = torch.randn(96, 300, generator=gen, device="cuda")
    dx, dw = torch.autograd.grad(z, (xg, w), dz)
    x8 = M8.dequantize(M8.quantize(x))
    y8 = M8.dequantize(M8.quantize(torch.sin(x)))
    assert torch.allclose(dx, (dz @ w.detach()) * torch.cos(x8), rtol=1e-4, atol=1e-4)
    assert torch.allclose(dw, dz.t() @ y8, rtol=1e-4, atol=1e-4)
    # shapes without long rows, another type, small tensors
    for shape in ((4000, 3), (7000,), (50, 40, 2)):
        t = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
        with M8.saved_tensors(min_elements=64):
            y = torch.sin(t * 1)
        assert torch.autograd.grad(y.sum(), t)[0].shape == t.shape
    small = torch.randn(10, generator=gen, device="cuda", requires_grad=True)
    with M8.saved_tensors(dtypes=(torch.float32, torch.bfloat16)):
        y = torch.sin(small * 1)
    assert torch.equal(torch.autograd.grad(y.sum(), small)[0], torch.cos(small.detach()))
    # float32 stays as it is unless asked for
    with M8.saved_tensors(min_elements=64):
        y = torch.sin(xg * 1.0)
    assert torch.equal(torch.autograd.grad(y, xg, torch.ones_like(y))[0], torch.cos(x))
    with pytest.raises(ValueError):
        M8.saved_tensors(dtypes=(torch.float16,))


@pytest.mark.parametrize("shape", [(30, 8, 40), (1 << 13, 32), (7, 11, 3, 5), (2000, 1), (96, 200)])
def test_saved_tensors_rows(shape):
    """Short last dimensions are joined with those before them, as one matrix: x itself, of x^2's gradient 2 x dy."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
    h = x * 1
    before = torch.cuda.memory_allocated()
    with M8.saved_tensors(min_elements=64):
        y = h * h
    held = torch.cuda.memory_allocated() - before - 2 * y.numel()
    cols = {(30, 8, 40): 320, (1 << 13, 32): 32, (7, 11, 3, 5): 165, (2000, 1): 2000, (96, 200): 200}[shape]
    # both factors' copies, each allocation rounded up to 512 bytes, as is y's
    assert held <= 2 * (x.numel() // cols * (cols + 31) // 32 * 33 + 512) + 512
    want = 2 * M8.dequantize(M8.quantize(x.detach().reshape(-1, cols)), torch.bfloat16).view(shape)
    assert torch.equal(torch.autograd.grad(y, x, torch.ones_like(y))[0], want)
    n = torch.complex(h.detach().float(), h.detach().float()).requires_grad_()
    m = (n * 1).conj().imag          # a view that negates what is in memory
    assert m.is_neg()
    with M8.saved_tensors(min_elements=64, dtypes=(torch.float32,)):
        y = m * m
    got = torch.autograd.grad(y, n, torch.ones_like(y))[0].imag
    assert torch.equal(got, 2 * M8.dequantize(M8.quantize(h.detach().float().reshape(-1, cols))).view(shape))


def test_saved_tensors_leave_what_a_matrix_cannot_hold():
    """Vectors of more than 2^29 elements stay as they are."""
    x = torch.ones((1 << 29) + 1, dtype=torch.bfloat16, device="cuda").requires_grad_()
    h = x * 3
    with M8.saved_tensors():
        y = h * h
    assert torch.equal(torch.autograd.grad(y.sum(), x)[0][-2:].float(), torch.full((2,), 18.0, device="cuda"))
