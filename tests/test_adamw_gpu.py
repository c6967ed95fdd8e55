"""The AdamW step and the gradient norm against the float64 oracle.

Tolerances (u = 2^-24): a moment takes three fp32 roundings, so it is within
4 u of the sum of its terms' magnitudes.  The update d = m / (sqrt(v) k + eps)
carries the relative errors of m (cancellation included), half of v's, and of a
square root, a reciprocal and the products around them: 16 u covers those; the
parameter adds three roundings of its own.  bf16 outputs add one spacing
(2^-7 relative, stochastic) or half of one (2^-8, to nearest).  An 8-bit code
may differ from the oracle's only where the moment's fp32 error, at most 2^-19
of a spacing of codes, crosses a rounding threshold: by one code, with
probability 2^-18 an element."""
import math

import numpy as np
import pytest
import torch

from oracle import adamw_mx4_oracle as O
from inverse_root_preconditioning_amd import adamw as AW
from inverse_root_preconditioning_amd import capi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _all(condition):
    return bool(np.all(condition))      # a failure prints no arrays


def _rng(*key):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(key)))


def _tensors(r, sizes, dtype, std, shift):
    """Tensors that begin `shift` elements into their storage (alignment of one element only)."""
    out = []
    for n in sizes:
        t = torch.zeros(n + shift, dtype=DT[dtype], device="cuda")[shift:]
        t.copy_(torch.from_numpy(r.standard_normal(n) * std))
        out.append(t)
    return out


def _flat(table_or_opt, tensors):
    """float64 copy of tensors in the state's layout."""
    flat = np.zeros(int(table_or_opt.offsets[-1]))
    for o, t in zip(table_or_opt.offsets, tensors):
        flat[o:o + t.numel()] = t.detach().double().cpu().numpy().reshape(-1)
    return flat


def _real(opt, sizes):
    real = np.zeros(int(opt.offsets[-1]), dtype=bool)
    for o, n in zip(opt.offsets, sizes):
        real[o:o + n] = True
    return real


def _values(opt):
    if opt.state == "f32":
        return opt.m.double().cpu().numpy(), opt.v.double().cpu().numpy()
    return (O.mx8_decode(opt.m.cpu().numpy(), opt.m_scale.cpu().numpy(), **O.M8),
            O.mx8_decode(opt.v.cpu().numpy(), opt.v_scale.cpu().numpy(), **O.V8))


def _ordered(code, fmt):
    """Codes as integers in the order of their values (both zeros are 0)."""
    c = code.astype(np.int64)
    return np.where(c >= 128, -(c & 127), c) if fmt["signed"] else c


SIZES = [1, 31, 32, 33, 0, 4095, 4096, 4097, 7, 10007, 64]


@pytest.mark.parametrize("param,grad,state,copy,shift", [
    ("f32", "f32", "f32", False, 0), ("f32", "f32", "f32", True, 1), ("f32", "bf16", "f32", True, 0),
    ("bf16", "bf16", "f32", False, 3), ("bf16", "f32", "f32", False, 0), ("f32", "f32", "mx8", False, 0),
    ("f32", "bf16", "mx8", True, 3), ("bf16", "bf16", "mx8", False, 0), ("bf16", "f32", "mx8", False, 1),
])
def test_three_steps_match_the_oracle(param, grad, state, copy, shift):
    print(f"adamw case: {param} {grad} {state} copy={copy} shift={shift}", flush=True)
    r = _rng(1, len(param), len(grad), len(state), shift)
    ps = _tensors(r, SIZES, param, 0.5, shift)
    cs = _tensors(r, SIZES, "bf16", 0.0, shift) if copy else None
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    scale = [1.0 + 0.5 * (i % 2) for i in range(len(SIZES))]
    opt = AW.AdamW(ps, weight_decay=decay, lr_scale=scale, state=state, copies=cs, seed=2 ** 40 + 7, **HYPER)
    real = _real(opt, SIZES)
    lr = np.zeros(real.size)
    wd = np.zeros(real.size)
    for o, n, a, b in zip(opt.offsets, SIZES, scale, decay):
        lr[o:o + n], wd[o:o + n] = 1e-2 * a, b
    b1, b2 = opt.betas
    for step in (1, 2, 3):
        gs = _tensors(r, SIZES, grad, 0.02 * 10.0 ** r.uniform(-2, 2), shift)
        p0, g = _flat(opt, ps), _flat(opt, gs)
        m0, v0 = _values(opt)
        coef = torch.tensor([0.75], device="cuda") if step == 2 else None
        opt.step(gs, grad_scale=coef)
        torch.cuda.synchronize()
        c = 0.75 if step == 2 else 1.0
        p1, m1, v1 = O.adamw(p0, g, m0, v0, lr, b1, b2, 1e-8, wd, step, c)
        tm = 4 * U * (b1 * np.abs(m0) + (1 - b1) * np.abs(g * c))
        tv = 4 * U * v1
        if state == "f32":
            m, v = _values(opt)
            assert _all(np.abs(m - m1)[real] <= tm[real] + 1e-44) and _all(np.abs(v - v1)[real] <= tv[real] + 1e-44)
        else:
            h = O.position_hash(np.arange(real.size), 2 ** 40 + 7, step)
            for name, x, h16, fmt in (("m", m1, h & np.uint64(0xFFFF), O.M8), ("v", v1, h >> np.uint64(16), O.V8)):
                want, ws = O.mx8_encode(np.where(real, x, 0.0), h16, **fmt)
                got = getattr(opt, name).cpu().numpy().astype(np.int64)
                gs8 = getattr(opt, name + "_scale").cpu().numpy()
                used = real.reshape(-1, 32).any(1)
                # the scale follows the largest magnitude's exponent, which the same error can move at a power of two
                top = np.abs(np.where(real, x, 0.0)).reshape(-1, 32).max(1)
                near = np.abs(top / 2.0 ** np.round(np.log2(np.maximum(top, 1e-300))) - 1) <= 4 * U
                assert _all((gs8 == ws)[used & ~near]), name
                same = np.repeat(gs8 == ws, 32)
                off = np.abs(_ordered(got, fmt) - _ordered(want, fmt))[real & same]
                assert off.max() <= 1 and off.astype(bool).sum() <= 3 + real.sum() * 2.0 ** -18, name
                apart = np.abs(O.mx8_decode(got, gs8, **fmt) - x)[real & ~same]
                assert _all(apart <= np.repeat(top, 32)[real & ~same] / 8), name
                assert _all(got[~real] == 0)
        d = (m1 / (1 - b1 ** step)) / (np.sqrt(v1 / (1 - b2 ** step)) + 1e-8)
        dm = tm / (1 - b1 ** step) / (np.sqrt(v1 / (1 - b2 ** step)) + 1e-8)
        tol = lr * (16 * U * np.abs(d) + dm) + 4 * U * (np.abs(p0) + np.abs(p1))
        got = _flat(opt, ps)
        if param == "bf16":
            tol = tol + 2.0 ** -7 * np.maximum(np.abs(p1), 2.0 ** -126)
        assert _all(np.abs(got - p1)[real] <= tol[real]), step
        if copy:
            assert np.array_equal(_flat(opt, cs), _flat(opt, [t.to(torch.bfloat16) for t in ps]))
    assert opt.t == 3


def test_a_table_of_no_elements_steps():
    for sizes in ([], [0], [0, 0]):
        opt = AW.AdamW(_tensors(_rng(2), sizes, "f32", 1.0, 0), state="mx8")
        g = AW.TensorTable(_tensors(_rng(2), sizes, "f32", 1.0, 0))
        opt.step(g)
        assert AW.grad_norm(g, 2.0).tolist() == [0.0, 1.0]
        assert opt.moments()[0].numel() == 0


@pytest.mark.parametrize("state", ["f32", "mx8"])
def test_extreme_gradients(state):
    """Zero, huge (v overflows fp32 to infinity) and tiny gradients, one group each, and a NaN."""
    n = 160
    g = torch.zeros(n, device="cuda")
    g[32:64] = 1e25
    g[64:96] = 1e-25
    g[96:128] = 1e-3
    g[128] = float("nan")
    p = torch.ones(n, device="cuda")
    opt = AW.AdamW([p], state=state, lr=0.1, weight_decay=0.0, betas=(0.9, 0.95))
    opt.step([g])
    q = p.cpu().numpy()
    m, v = (t.cpu().numpy() for t in opt.moments())
    assert _all(q[:32] == 1) and _all(np.isfinite(q[:32]))
    assert _all(np.abs(q[96:128] - 0.9) < 1e-4)          # the first step is lr in size (eps / |g| is 1e-5)
    assert _all(np.abs(1 - q[64:96]) < 1e-6)             # |g| far below eps
    assert np.isnan(q[128]) and _all(q[129:] == 1)
    if state == "f32":
        assert _all(np.isinf(v[32:64])) and np.isnan(m[128]) and _all(m[129:] == 0)
    else:
        assert _all(np.isnan(v[32:64])) and _all(np.isnan(m[128:]))
        assert _all(m[:32] == 0) and _all(v[:32] < 1e-40)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_scale_that_is_not_finite_changes_nothing(value):
    r = _rng(3)
    ps, gs = _tensors(r, [100, 5000], "f32", 1.0, 0), _tensors(r, [100, 5000], "f32", 1.0, 0)
    opt = AW.AdamW(ps, state="mx8")
    opt.step(gs)
    before = [t.clone() for t in (*ps, opt.m, opt.v, opt.m_scale, opt.v_scale)]
    opt.step(gs, grad_scale=torch.full((1,), value, device="cuda"))
    for a, b in zip(before, (*ps, opt.m, opt.v, opt.m_scale, opt.v_scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("param,state", [("f32", "mx8"), ("bf16", "mx8"), ("bf16", "f32")])
def test_same_seed_same_bits_and_resume(param, state):
    def run(seed, resume):
        r = _rng(4)
        sizes = [333, 4097, 50]
        ps = _tensors(r, sizes, param, 1.0, 0)
        opt = AW.AdamW(ps, state=state, seed=seed)
        for t in range(4):
            if resume and t == 2:
                saved = {k: v.clone() if torch.is_tensor(v) else v for k, v in opt.state_dict().items()}
                opt = AW.AdamW(ps, state=state, seed=0)
                opt.load_state_dict(saved)
            opt.step(_tensors(r, sizes, "f32", 0.1, 0))
        return [t.clone() for t in (*ps, opt.m, opt.v)]
    a, b, c, d = run(1, False), run(1, False), run(1, True), run(2, False)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and all(torch.equal(x, y) for x, y in zip(a, c))
    assert not all(torch.equal(x, y) for x, y in zip(a, d))


def test_stochastic_rounding_keeps_small_changes_on_average():
    """v = 1 and m = 1 in every entry; each step changes them by less than a
    spacing of codes.  After k steps the mean over n entries follows the exact
    average; its standard error is at most a spacing over sqrt(n) times
    sqrt(k).  A bf16 parameter moves by 2^-12 a step, below half its spacing."""
    n, k = 1 << 16, 20
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    opt = AW.AdamW([p], lr=2.0 ** -12, betas=(0.99, 0.999), eps=0.0, weight_decay=0.0, state="mx8", seed=9)
    g = torch.ones(n, device="cuda")
    opt.step([g])
    opt.t = 10 ** 7                          # no bias correction
    m0, v0 = (t.double().mean().item() for t in opt.moments())
    for _ in range(k):
        opt.step([g])
    m, v = (t.double().mean().item() for t in opt.moments())
    em, ev = 1 - (1 - m0) * 0.99 ** k, 1 - (1 - v0) * 0.999 ** k
    assert abs(m - em) <= 6 * em / 8 * math.sqrt(k / n) and abs(v - ev) <= 6 * ev / 8 * math.sqrt(k / n)
    assert p.float().mean().item() < 1       # it moved


def test_states_in_8_bits_train_like_states_in_32():
    """A least-squares problem reaches the same loss within a fifth of the start's distance."""
    r = _rng(5)
    a = torch.from_numpy(r.standard_normal((512, 256)) / 16).float().cuda()
    y = a @ torch.from_numpy(r.standard_normal(256)).float().cuda()
    loss = {}
    for state in ("f32", "mx8"):
        w = torch.zeros(256, device="cuda")
        opt = AW.AdamW([w], lr=2e-2, betas=(0.9, 0.99), weight_decay=0.0, state=state)
        for _ in range(400):
            opt.step([a.t() @ (a @ w - y)])
        loss[state] = (a @ w - y).square().sum().item()
    start = y.square().sum().item()
    assert loss["f32"] < 0.01 * start and loss["mx8"] < 0.01 * start


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_moments_are_the_oracles_values(dtype):
    r = _rng(6)
    opt = AW.AdamW(_tensors(r, [1000, 4096], "f32", 1.0, 0), state="mx8")
    opt.m.copy_(torch.from_numpy(r.integers(0, 256, opt.m.numel())))
    opt.v.copy_(torch.from_numpy(r.integers(0, 256, opt.v.numel())))
    opt.m_scale.copy_(torch.from_numpy(r.integers(30, 220, opt.m_scale.numel())))
    opt.v_scale.copy_(torch.from_numpy(r.integers(30, 220, opt.v_scale.numel())))
    opt.m_scale[3] = 255
    for got, want in zip(opt.moments(DT[dtype]), _values(opt)):
        assert got.dtype == DT[dtype] and np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


# ---------------------------------------------------------------------------
# The norm
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,shift", [("f32", 0), ("f32", 1), ("bf16", 0), ("bf16", 5)])
@pytest.mark.parametrize("sizes", [[1], [0, 3], SIZES, [1 << 20] * 9 + [12345]])
def test_norm_and_coefficient(dtype, shift, sizes):
    """Squares are exact in double and their sum is off by less than 1e-12; the outputs are rounded once to fp32."""
    print(f"norm case: {dtype} {shift} {len(sizes)}", flush=True)
    ts = _tensors(_rng(7, shift), sizes, dtype, 0.3, shift)
    table = AW.TensorTable(ts)
    n, _ = O.grad_norm([t.double().cpu().numpy() for t in ts], 1.0)
    for limit in (0.5 * n, 2 * n, math.inf):
        got = AW.grad_norm(table, limit).tolist()
        want = 1.0 if limit >= n else float(np.float32(limit)) / n
        assert abs(got[0] - n) <= 2 * U * n and abs(got[1] - want) <= 2 * U
    again = AW.grad_norm(table, 1.0), AW.grad_norm(table, 1.0)
    assert torch.equal(*again)


def test_norm_of_extreme_entries():
    big = torch.full((5000,), 1e37, device="cuda")      # the norm, 7e38, is above fp32's range
    got = AW.grad_norm(AW.TensorTable([big]), 1.0).tolist()
    assert math.isinf(got[0]) and math.isnan(got[1])
    got = AW.grad_norm(AW.TensorTable([big[:1000]]), 1.0).tolist()   # 3.2e38 is within it
    assert abs(got[0] / (1e37 * math.sqrt(1000)) - 1) < 1e-6 and 0 < got[1] < 1e-38
    small = torch.full((100,), 1e-30, device="cuda")
    assert abs(AW.grad_norm(AW.TensorTable([small]), 1.0)[0].item() / 1e-29 - 1) < 1e-6
    for value in (float("nan"), float("inf")):
        big[17] = value
        out = AW.grad_norm(AW.TensorTable([big]), 1.0)
        assert not math.isfinite(out[0].item()) and math.isnan(out[1].item())


# ---------------------------------------------------------------------------
# Streams, graphs, refusals
# ---------------------------------------------------------------------------

def test_on_a_side_stream():
    r = _rng(8)
    sizes = [5000, 123]
    results = []
    for side in (False, True):
        r = _rng(8)
        ps, gs = _tensors(r, sizes, "f32", 1.0, 0), _tensors(r, sizes, "bf16", 1.0, 0)
        opt, table = AW.AdamW(ps, state="mx8"), AW.TensorTable(gs)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream() if side else None
        for _ in range(3):
            norm = AW.grad_norm(table, 1.0, stream=stream)
            opt.step(table, grad_scale=norm[1:], stream=stream)
        m, v = opt.moments(stream=stream)
        torch.cuda.synchronize()
        results.append([t.clone() for t in (*ps, m, v, norm)])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_captured_step_replays_like_eager():
    """A graph holds one step's bias correction, so the eager runs repeat that step count."""
    r = _rng(9)
    sizes = [3000, 4096, 17]
    init = _tensors(r, sizes, "f32", 1.0, 0)
    pairs = []
    for _ in range(2):
        ps = [t.clone() for t in init]
        pairs.append((ps, AW.AdamW(ps, state="mx8", seed=3)))
    gs = _tensors(r, sizes, "f32", 0.1, 0)
    table = AW.TensorTable(gs)
    (pe, eager), (pg, graphed) = pairs
    warm = AW.grad_norm(table, 1.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = AW.grad_norm(table, 1.0)
        graphed.step(table, grad_scale=norm[1:])
    for i in range(4):
        for g in gs:
            g.mul_(1.5)
        eager.t = 0
        eager.step(table, grad_scale=AW.grad_norm(table, 1.0)[1:])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(pe, pg)), i
        assert torch.equal(eager.m, graphed.m) and torch.equal(eager.v_scale, graphed.v_scale), i
    assert torch.isfinite(warm).all()


def test_refusals():
    f = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="one type"):
        AW.TensorTable([f, f.bfloat16()])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        AW.TensorTable([f.half()])
    with pytest.raises(ValueError, match="CUDA"):
        AW.TensorTable([f.cpu()])
    with pytest.raises(ValueError, match="not dense"):
        AW.TensorTable([f[::2]])
    with pytest.raises(ValueError, match="not dense"):
        AW.TensorTable([f[:1].expand(8)])
    AW.TensorTable([torch.zeros(8, 4, device="cuda").t()])
    opt = AW.AdamW([f], state="mx8")
    with pytest.raises(ValueError, match="differ from the parameters"):
        opt.step([f[:32]])
    with pytest.raises(ValueError, match="differ from the parameters"):
        AW.AdamW([torch.zeros(8, 4, device="cuda")]).step([torch.zeros(4, 8, device="cuda").t()])
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step([f], grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="state"):
        AW.AdamW([f], state="f16")
    with pytest.raises(ValueError, match="betas"):
        AW.AdamW([f], betas=(1.0, 0.9))
    with pytest.raises(ValueError, match="weight_decay"):
        AW.AdamW([f], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError, match="copies"):
        AW.AdamW([f], copies=[f])
    with pytest.raises(ValueError, match="another kind"):
        opt.load_state_dict(AW.AdamW([f]).state_dict())
    with pytest.raises(capi.ShampooError):
        opt.step([f], lr=float("nan"))
    with pytest.raises(capi.ShampooError):
        AW.grad_norm(AW.TensorTable([f]), 0.0)
