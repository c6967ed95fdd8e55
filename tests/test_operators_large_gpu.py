"""Offsets beyond 32 bits and other extremes of size of the AdamW, norm and MX4
operators, checked at places where a truncated offset would show."""
import numpy as np
import pytest
import torch

from oracle import adamw_mx4_oracle as O
from inverse_root_preconditioning_amd import adamw as AW
from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx4 as MX

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _f64(t):
    return t.detach().double().cpu().numpy()


def test_adamw_and_norm_of_more_than_2_to_32_elements():
    """Two bf16 tensors, the second's state beyond position 2^32.  Zero gradients
    except at the ends: only there do parameters move, and the hash uses the
    upper half of the position."""
    n = (1 << 32) + 4099
    sizes = [n, 70]
    ps = [torch.zeros(k, dtype=torch.bfloat16, device="cuda") for k in sizes]
    gs = [torch.zeros(k, dtype=torch.bfloat16, device="cuda") for k in sizes]
    opt = AW.AdamW(ps, lr=1.0, weight_decay=0.0, betas=(0.9, 0.95), state="mx8", seed=5)
    gs[0][-40:] = 3.0
    gs[0][:5] = -2.0
    gs[1][:] = 0.5
    table = AW.TensorTable(gs)
    norm = AW.grad_norm(table, 1e9)[0].item()
    assert abs(norm - (40 * 9.0 + 5 * 4.0 + 70 * 0.25) ** 0.5) < 1e-4
    opt.step(table)
    torch.cuda.synchronize()
    # the first step is lr against the gradient's sign, within a bf16 spacing
    assert torch.all((ps[0][-40:].float() + 1).abs() <= 2.0 ** -7) and torch.all((ps[0][:5].float() - 1).abs() <= 2.0 ** -7)
    assert torch.all((ps[1].float() + 1).abs() <= 2.0 ** -7)
    assert int(torch.count_nonzero(ps[0])) == 45
    first = int(opt.offsets[1])
    pos = first + np.arange(64)
    h = O.position_hash(pos, 5, 1)
    m = np.full(64, (1 - 0.9) * 0.5)
    want, ws = O.mx8_encode(m, h & np.uint64(0xFFFF), **O.M8)
    got = opt.m[first:first + 64].cpu().numpy()
    assert np.array_equal(opt.m_scale[first // 32:first // 32 + 2].cpu().numpy(), ws) and np.abs(
        got.astype(int) - want.astype(int)).max() <= 1 and (got != want).sum() <= 1


def test_quantise_and_dequantise_beyond_32_bit_offsets():
    rows, cols = 70000, 65536                       # 4.6e9 elements
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    places = [0, 1, 32767, 32768, 65535, 65536, rows - 1]
    r = np.random.Generator(np.random.PCG64(1))
    for k in places:
        x[k] = torch.from_numpy(r.standard_normal(cols)).cuda()
    q, qt = MX.quantize_both(x)
    v = MX.dequantize(q, torch.bfloat16)
    for k in places:
        assert np.array_equal(_f64(v[k:k + 1]), O.mx4_round(_f64(x[k:k + 1])))
    del v, q
    v = MX.dequantize(qt, torch.bfloat16)
    for c in (0, 40000, cols - 1):
        assert np.array_equal(_f64(v[c:c + 1]), O.mx4_round(_f64(x[:, c:c + 1]).T))


def test_product_with_an_output_beyond_32_bit_offsets():
    M, N, K = 70000, 65600, 64                      # C: 4.6e9 elements
    r = np.random.Generator(np.random.PCG64(2))
    a = MX.quantize(torch.from_numpy(r.standard_normal((M, K))).float().cuda())
    b = MX.quantize(torch.from_numpy(r.standard_normal((N, K))).float().cuda())
    c = MX.product(a, b, dtype=torch.bfloat16)
    av, bv = _f64(MX.dequantize(a)), _f64(MX.dequantize(b))
    for rows in (slice(0, 3), slice(65470, 65475), slice(M - 3, M)):
        want = av[rows] @ bv.T
        tol = (K + 8) * 2.0 ** -24 * (np.abs(av[rows]) @ np.abs(bv).T) + 2.0 ** -8 * np.abs(want)
        assert bool(np.all(np.abs(_f64(c[rows]) - want) <= tol))


@pytest.mark.parametrize("M,N,K,dtype,beta", [
    (4400, 4300, 1000, "f32", 0.0), (4400, 4301, 2048, "bf16", 0.0), (6001, 6000, 1024, "bf16", 0.0),
    (4096, 4352, 5000, "f32", 0.0), (70001, 255, 1024, "f32", 0.0), (4400, 4300, 1000, "f32", 0.5), (4400, 4300, 1100, "bf16", 0.0)])
def test_product_of_more_tiles_than_compute_units(M, N, K, dtype, beta):
    """Workgroups that go from tile to tile, whole ones and those at the edges,
    once to three times, into rows that lie further apart than they are long."""
    print(f"tiles case: {M} {N} {K} {dtype} {beta}", flush=True)
    r = np.random.Generator(np.random.PCG64([M, N, K]))
    a = MX.quantize(torch.from_numpy(r.standard_normal((M, K), dtype=np.float32)).cuda())
    b = MX.quantize(torch.from_numpy(r.standard_normal((N, K), dtype=np.float32)).cuda())
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    whole = torch.full((M, N + 24), 0.75, device="cuda", dtype=td)
    out = whole[:, 8:N + 8]
    MX.product(a, b, out=out, alpha=-0.5, beta=beta)
    av, bv = MX.dequantize(a).double(), MX.dequantize(b).double().T.contiguous()
    want = -0.5 * (av @ bv) + beta * 0.75
    tol = (K + 8) * 2.0 ** -24 * (0.5 * (av.abs() @ bv.abs()) + beta * 0.75)
    if dtype == "bf16":
        tol += 2.0 ** -8 * want.abs()
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool((whole[:, :8] == 0.75).all()) and bool((whole[:, N + 8:] == 0.75).all())
    first = whole.clone()
    if beta == 0.0:
        for _ in range(3):                          # the same bits again
            MX.product(a, b, out=out, alpha=-0.5)
            assert torch.equal(whole, first)


@pytest.mark.parametrize("M,N", [(20, 5), (300, 300)])
def test_product_over_no_columns(M, N):
    z = lambda r: MX.quantize(torch.zeros(r, 0, device="cuda"))  # noqa: E731
    out = torch.full((M, N), 3.0, device="cuda")
    assert torch.all(MX.product(z(M), z(N), out=out, beta=0.5) == 1.5)
    assert torch.all(MX.product(z(M), z(N), dtype=torch.float32) == 0)


def test_train_linear_refuses_a_second_derivative():
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    w = torch.randn(16, 64, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(MX.train_linear(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
