"""MX4 quantisation and products against the float64 oracle.

Quantised codes and scales are compared exactly (every rounding is defined).
Products: the terms are exact in fp32, so a result is within (K + 8) 2^-24 of
the sum of the terms' magnitudes of the exact one, plus half a spacing of bf16
(2^-8 relative) where it is rounded to that, and 2^-23 of each of alpha AB and
beta C."""
import numpy as np
import pytest
import torch

from oracle import adamw_mx4_oracle as O
from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx4 as MX

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _all(condition):
    return bool(np.all(condition))      # a failure prints no arrays


def _rng(*key):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(key)))


def _input(r, rows, cols, dtype, std=1.0):
    x = r.standard_normal((rows, cols)) * std * np.exp(r.standard_normal(cols))
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _codes(q):
    """(4-bit codes, scales) of an MX4Matrix, columns padded to 32 only; the rest checked to be zero codes."""
    b = q.codes.cpu().numpy()
    c = np.stack([b & 15, b >> 4], axis=2).reshape(q.rows, -1)
    w = -(-q.cols // 32) * 32
    assert _all(c[:, q.cols:] == 0)
    return c[:, :w], q.scales.cpu().numpy()[:, :w // 32]


def _check_codes(q, x):
    code, scale = O.mx4_quantize(x)
    got, gs = _codes(q)
    assert np.array_equal(gs, scale)
    assert np.array_equal(got & 7, code & 7)
    assert np.array_equal(got[(code & 7) > 0], code[(code & 7) > 0])      # the sign of a zero is free


SHAPES = [(1, 1), (1, 2048), (3, 31), (5, 33), (128, 128), (129, 127), (257, 300), (64, 1001), (1000, 65), (31, 4096),
          (2049, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_both_ways(rows, cols, dtype):
    print(f"quantise case: {rows}x{cols} {dtype}", flush=True)
    x = _input(_rng(1, rows, cols), rows, cols, dtype)
    q, qt = MX.quantize_both(x)
    _check_codes(q, _f64(x))
    _check_codes(qt, _f64(x).T)
    assert torch.equal(MX.quantize(x).codes, q.codes) and torch.equal(MX.quantize(x.t()).codes, qt.codes)
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(_f64(MX.dequantize(q, out)), O.mx4_round(_f64(x)))
        assert np.array_equal(_f64(MX.dequantize(qt, out)), O.mx4_round(_f64(x).T))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_every_value_at_ties_and_scales(dtype):
    """All multiples of a quarter spacing around every code, over the whole range of exponents."""
    base = np.concatenate([np.arange(0, 8, 0.125), -np.arange(0, 8, 0.125)])
    rows = [np.concatenate([[4.0], np.resize(base[i:], 31)]) * 2.0 ** e for e in (-126, -120, -1, 0, 40, 124)
            for i in range(0, 128, 31)]
    x = torch.from_numpy(np.stack(rows)).to(DT[dtype]).cuda()
    q, qt = MX.quantize_both(x)
    _check_codes(q, _f64(x))
    _check_codes(qt, _f64(x).T)


def test_quantize_special_groups():
    x = torch.zeros(40, 256, device="cuda")
    x[0, 3] = float("nan")
    x[1, 40] = float("inf")
    x[2, 70] = -float("inf")
    x[3, 100] = 1e-40
    x[4, 130] = torch.finfo(torch.float32).max
    x[5] = torch.finfo(torch.float32).tiny
    q, qt = MX.quantize_both(x)
    _check_codes(q, _f64(x))
    _check_codes(qt, _f64(x).T)
    v = MX.dequantize(q)
    assert torch.isnan(v[0, :32]).all() and not torch.isnan(v[0, 32:]).any() and torch.isnan(v[1, 32:64]).all()


def test_quantize_of_strided_rows():
    r = _rng(2)
    for dtype in ("f32", "bf16"):
        for start, cols, ld in ((0, 100, 131), (1, 96, 97), (8, 128, 264), (3, 33, 200)):
            big = _input(r, 70, ld, dtype)
            x = big[:, start:start + cols]
            q, qt = MX.quantize_both(x)
            _check_codes(q, _f64(x))
            _check_codes(qt, _f64(x).T)


def _product_case(M, N, K, dtype, alpha, beta, key):
    r = _rng(3, key, M, N, K)
    a, b = MX.quantize(_input(r, M, K, "f32")), MX.quantize(_input(r, N, K, "f32"))
    big = torch.from_numpy(r.standard_normal((M, N + 5))).to(DT[dtype]).cuda()
    c = big[:, 2:N + 2]                                       # strided and misaligned output
    if beta == 0.0:
        c.fill_(float("nan"))
    before, around = _f64(c), big.clone()
    av, bv = _f64(MX.dequantize(a)), _f64(MX.dequantize(b))
    MX.product(a, b, out=c, alpha=alpha, beta=beta)
    torch.cuda.synchronize()
    want = alpha * (av @ bv.T) + (beta * before if beta else 0.0)
    mag = abs(alpha) * (np.abs(av) @ np.abs(bv).T)
    tol = (K + 8) * 2.0 ** -24 * mag + 2.0 ** -23 * (np.abs(want) + abs(beta) * np.abs(np.nan_to_num(before)))
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want)
    got = _f64(c)
    assert _all(np.abs(got - want) <= tol + 1e-40), (np.abs(got - want) / (tol + 1e-40)).max()
    assert torch.equal(big[:, :2], around[:, :2]) and torch.equal(big[:, N + 2:], around[:, N + 2:])


PRODUCTS = [(1, 1, 1), (1, 17, 33), (16, 16, 128), (1, 1000, 2048), (7, 130, 300), (33, 65, 1000), (100, 100, 100),
            (128, 128, 512), (257, 255, 129), (300, 513, 1537), (512, 256, 4096), (1, 4096, 64), (2000, 3, 200),
            (15, 2048, 8192), (40, 1024, 2048), (640, 768, 1024), (1030, 1027, 260), (17, 64, 4096),
            (100, 300, 5000), (64, 2048, 8192), (333, 129, 12345), (16, 8200, 1200), (3, 8192, 2049)]


@pytest.mark.parametrize("dtype,alpha,beta", [("f32", 1.0, 0.0), ("bf16", 1.0, 0.0), ("f32", -0.5, 1.0),
                                              ("bf16", 2.0, 0.25)])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, dtype, alpha, beta):
    print(f"product case: {M} {N} {K} {dtype} {alpha} {beta}", flush=True)
    _product_case(M, N, K, dtype, alpha, beta, 0)


def test_product_of_empty_matrices():
    z = lambda r, c: MX.quantize(torch.zeros(r, c, device="cuda"))  # noqa: E731
    assert MX.product(z(0, 64), z(5, 64)).shape == (0, 5)
    assert MX.product(z(4, 64), z(0, 64)).shape == (4, 0)
    out = torch.full((4, 5), 3.0, device="cuda")
    MX.product(z(4, 0), z(5, 0), out=out, beta=0.5)
    assert torch.all(out == 1.5)
    assert torch.all(MX.product(z(4, 0), z(5, 0), dtype=torch.float32) == 0)
    assert MX.linear(torch.zeros(2, 0, 64, device="cuda"), z(5, 64)).shape == (2, 0, 5)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_nan_groups_reach_their_row_and_column_only(M):
    r = _rng(4)
    x, w = _input(r, M, 256, "f32"), _input(r, 200, 256, "f32")
    x[0, 100], w[7, 3] = float("inf"), float("nan")
    c = MX.product(MX.quantize(x), MX.quantize(w), dtype=torch.float32)
    want = torch.zeros(M, 200, dtype=torch.bool, device="cuda")
    want[0, :], want[:, 7] = True, True
    assert torch.equal(torch.isnan(c), want)


def test_product_is_exact_over_the_whole_scale_range():
    """Groups whose scales differ by 2^40 and more: powers of two, so that every sum is exact."""
    M, N, K = 48, 80, 384
    r = _rng(5)
    x = np.zeros((M, K))
    for g in range(K // 32):
        x[:, 32 * g + g % 32] = 2.0 ** (5 * g - 30)
    w = np.zeros((N, K))
    pick = r.integers(0, K // 32, N)
    for j in range(N):
        w[j, 32 * pick[j] + pick[j] % 32] = 2.0 ** (j - 40)
    c = MX.product(MX.quantize(torch.from_numpy(x).float().cuda()), MX.quantize(torch.from_numpy(w).float().cuda()),
                   dtype=torch.float32)
    assert np.array_equal(_f64(c), x @ w.T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 8192, 2048), (1, 5, 7), (2, 100, 2048), (13, 333, 1001), (16, 256, 4096),
                                   (17, 300, 8192), (64, 640, 130), (200, 1000, 520)])
def test_linear_is_the_product_of_the_quantised_input(M, N, K, dtype):
    """Bits equal to the two calls where both take the same form; else within the product's tolerance."""
    print(f"linear case: {M} {N} {K} {dtype}", flush=True)
    r = _rng(6, M, N, K)
    x, w = _input(r, M, K, dtype), MX.quantize(_input(r, N, K, "f32", 0.1))
    y = MX.linear(x, w)
    xv, wv = O.mx4_round(_f64(x)), _f64(MX.dequantize(w))
    want = xv @ wv.T
    tol = (K + 8) * 2.0 ** -24 * (np.abs(xv) @ np.abs(wv).T) + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -23) * np.abs(want)
    assert y.dtype == x.dtype and _all(np.abs(_f64(y) - want) <= tol + 1e-40)
    if M > 1:
        pad = torch.cat([x, x], dim=1)
        assert torch.equal(MX.linear(pad[:, :K], w), y)              # strided rows
        assert torch.equal(MX.linear(x.view(M, 1, K), w).view(M, N), y)
    out = torch.zeros(M, N, dtype=x.dtype, device="cuda")
    assert torch.equal(MX.linear(x, w, out=out), y) and torch.equal(out, y)


@pytest.mark.parametrize("xt,wt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (3, 40, 70), (130, 257, 96), (512, 256, 384)])
def test_train_linear_gradients_are_the_formulas(T, N, K, xt, wt):
    print(f"train case: {T} {N} {K} {xt} {wt}", flush=True)
    r = _rng(7, T, N, K)
    x, w, dy = _input(r, T, K, xt), _input(r, N, K, wt, 0.1), _input(r, T, N, xt, 1e-3)
    x.requires_grad_(), w.requires_grad_()
    y = MX.train_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    X, W, D = _f64(x), _f64(w), _f64(dy)
    for got, a, b in ((y, O.mx4_round(X), O.mx4_round(W)), (dx, O.mx4_round(D), O.mx4_round(W.T)),
                      (dw, O.mx4_round(D.T), O.mx4_round(X.T))):
        want = a @ b.T
        tol = (a.shape[1] + 8) * 2.0 ** -24 * (np.abs(a) @ np.abs(b).T)
        tol = tol + (2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(want)
        assert _all(np.abs(_f64(got) - want) <= tol + 1e-40)


def test_train_linear_gradients_are_differences():
    """Inputs that MX4 holds exactly along both dimensions (magnitudes 1 to 6 in
    every group): there the quantisers are the identity, the loss is bilinear,
    and a central difference between two such inputs is the gradient times the
    step."""
    r = _rng(8)
    T, N, K = 32, 64, 96
    grid = np.array([1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    pick = lambda *s: grid[r.integers(0, 6, s)] * r.choice([-1.0, 1.0], s)  # noqa: E731

    def fix(a):                      # a 4 in every group both ways fixes all scales
        a[::32, :] = 4.0
        a[:, ::32] = 4.0
        return a
    X, W, D = fix(pick(T, K)), fix(pick(N, K)), fix(pick(T, N))
    dev = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    x, w, dy = dev(X).requires_grad_(), dev(W).requires_grad_(), dev(D)
    dx, dw = torch.autograd.grad(MX.train_linear(x, w), (x, w), dy)
    loss = lambda a, b: float((_f64(MX.train_linear(dev(a), dev(b))) * D).sum())  # noqa: E731
    for i, k in ((5, 7), (31, 95), (17, 40)):
        up, down = X.copy(), X.copy()
        up[i, k], down[i, k] = 6.0, -6.0
        assert abs((loss(up, W) - loss(down, W)) / 12 - dx[i, k].item()) <= 1e-5 * (abs(dx[i, k].item()) + 1)
    for n, k in ((5, 7), (63, 95), (40, 33)):
        up, down = W.copy(), W.copy()
        up[n, k], down[n, k] = 6.0, -6.0
        assert abs((loss(X, up) - loss(X, down)) / 12 - dw[n, k].item()) <= 1e-5 * (abs(dw[n, k].item()) + 1)


def test_train_linear_leading_dimensions_and_partial_gradients():
    r = _rng(9)
    x, w = _input(r, 6, 64, "f32").view(2, 3, 64), _input(r, 40, 64, "f32")
    y0 = MX.train_linear(x, w)
    x.requires_grad_()
    y = MX.train_linear(x, w)
    assert y.shape == (2, 3, 40) and torch.equal(y, y0)
    y.sum().backward()                                        # an expanded gradient
    assert x.grad.shape == x.shape and w.grad is None
    w.requires_grad_()
    x2 = x.detach()
    MX.train_linear(x2, w).sum().backward()
    assert w.grad.shape == w.shape and torch.isfinite(w.grad).all()


def test_on_a_side_stream_and_in_a_graph():
    r = _rng(10)
    x, w = _input(r, 40, 640, "bf16"), MX.quantize(_input(r, 300, 640, "f32"))
    x1 = x[:1].clone()
    want, want1 = MX.linear(x, w), MX.linear(x1, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, got1 = MX.linear(x, w, stream=s), MX.linear(x1, w, stream=s)
    q = MX.quantize(x, stream=s)
    p = MX.product(q, w, stream=s)
    d = MX.dequantize(q, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got1, want1) and torch.equal(p, want)
    assert np.array_equal(_f64(d), O.mx4_round(_f64(x)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        yg, y1 = MX.linear(x, w), MX.linear(x1, w)
    for i in range(4):
        x.mul_(0.75)
        x1.add_(0.5)
        eager, eager1 = MX.linear(x, w), MX.linear(x1, w)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, eager) and torch.equal(y1, eager1), i


def test_repeated_calls_give_the_same_bits():
    r = _rng(11)
    for M, N, K in ((1, 4096, 4096), (9, 512, 8192), (500, 700, 3001)):
        x, w = _input(r, M, K, "bf16"), MX.quantize(_input(r, N, K, "f32"))
        a = MX.linear(x, w)
        for _ in range(3):
            assert torch.equal(MX.linear(x, w), a)


def test_refusals():
    x = torch.zeros(8, 64, device="cuda")
    q = MX.quantize(x)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        MX.quantize(x.half())
    with pytest.raises(ValueError, match="CUDA"):
        MX.quantize(x.cpu())
    with pytest.raises(ValueError, match="contiguous rows"):
        MX.quantize(torch.zeros(8, 64, 2, device="cuda")[:, :, 0])
    with pytest.raises(ValueError, match="two dimensions"):
        MX.quantize(x[0])
    with pytest.raises(ValueError, match="overlap"):
        MX.quantize(x[:1].expand(8, 64))
    with pytest.raises(ValueError, match="columns"):
        MX.product(q, MX.quantize(torch.zeros(8, 65, device="cuda")))
    with pytest.raises(ValueError, match="beta needs out"):
        MX.product(q, q, beta=1.0)
    with pytest.raises(ValueError, match="shape"):
        MX.product(q, q, out=torch.zeros(8, 9, device="cuda"))
    with pytest.raises(ValueError, match="columns"):
        MX.linear(torch.zeros(3, 65, device="cuda"), q)
    with pytest.raises(ValueError, match="do not multiply"):
        MX.train_linear(x, torch.zeros(4, 65, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        MX.MX4Matrix(q.codes, q.scales, 8, 200)
    with pytest.raises(ValueError, match="uint8"):
        MX.MX4Matrix(q.codes.float(), q.scales, 8, 64)
    with pytest.raises(ValueError, match="aligned"):
        MX.MX4Matrix(torch.zeros(8 * 64 + 1, dtype=torch.uint8, device="cuda")[1:].view(8, 64), q.scales, 8, 64)
    with pytest.raises(capi.ShampooError):
        MX.product(q, q, alpha=float("inf"))
