"""What the AdamW object keeps, saves and refuses, and the edges of its arithmetic."""
import io
import math
import weakref

import numpy as np
import pytest
import torch

from oracle import adamw_mx4_oracle as O
from inverse_root_preconditioning_amd import adamw as AW
from inverse_root_preconditioning_amd import capi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def test_gradients_are_not_kept_after_the_step():
    p = [torch.zeros(1000, device="cuda"), torch.zeros(50, device="cuda")]
    opt = AW.AdamW(p)
    for as_table in (False, True):
        g = [torch.ones_like(t) for t in p]
        refs = [weakref.ref(t) for t in g]
        if as_table:
            table = AW.TensorTable(g)
            opt.step(table)
            opt.step(table)
            del table
        else:
            opt.step(g)
        del g
        assert all(r() is None for r in refs), as_table


def test_tables_are_checked_after_another_was():
    p = [torch.zeros(64, device="cuda"), torch.zeros(32, device="cuda")]
    opt = AW.AdamW(p)
    opt.step([torch.ones_like(t) for t in p])
    with pytest.raises(ValueError, match="differ from the parameters"):
        opt.step([torch.ones_like(t) for t in reversed(p)])
    opt.step([torch.ones_like(t) for t in p])
    assert opt.t == 2


@pytest.mark.parametrize("state", ["f32", "mx8"])
@pytest.mark.parametrize("size", [1e-19, 1e-20, 1e-21])
def test_second_moments_below_the_normal_range(size, state):
    """eps = 0: the first step is lr in size whatever the gradient's.  v lies in
    fp32's subnormals, 2^-149 apart, and is rounded to them: its relative error
    is at most 2^-150 / v, half of it the update's."""
    p = torch.ones(96, device="cuda")
    opt = AW.AdamW([p], lr=0.125, betas=(0.9, 0.95), eps=0.0, weight_decay=0.0, state=state)
    g = torch.full((96,), size, device="cuda")
    g[::2] *= -1
    opt.step([g])
    v = 0.05 * float(g.abs()[0]) ** 2
    tol = 0.125 * (2.0 ** -150 / v + 32 * U) + 2 * U
    want = torch.where(g > 0, 0.875, 1.125).double()
    off = (p.double() - want).abs().max().item()
    assert off <= tol


@pytest.mark.parametrize("eps", [1e-38, 1e-40, 1e-50])
def test_an_eps_below_the_normal_range_divides_zero(eps):
    """A gradient of 0 leaves m = v = 0, and 0 / eps is 0."""
    p = torch.ones(96, device="cuda")
    opt = AW.AdamW([p], lr=0.125, eps=eps, weight_decay=0.0)
    g = torch.zeros(96, device="cuda")
    g[5] = 1.0
    opt.step([g])
    assert p[5].item() == 0.875 and p.sum().item() == 95.875


def test_parameters_that_share_memory_are_refused():
    """Two workgroups would update the same elements."""
    flat = torch.zeros(200, device="cuda")
    for bad in ([flat, flat], [flat[:40], flat[32:64]], [flat[100:], flat[:50], flat[40:60]]):
        with pytest.raises(ValueError, match="share memory"):
            AW.AdamW(bad)
    opt = AW.AdamW([flat[100:], flat[:40], flat[40:60], flat[:0], flat[60:60]])   # apart from one another
    opt.step([torch.ones(n, device="cuda") for n in (100, 40, 20, 0, 0)])
    p = [torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")]
    c = torch.zeros(100, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="share memory"):
        AW.AdamW(p, copies=[c[:64], c[36:]])
    with pytest.raises(ValueError, match="share memory"):
        AW.AdamW(p, copies=[p[0].view(torch.bfloat16)[:64], c[:64]])
    # gradients are only read: tied ones may be one tensor
    g = torch.ones(64, device="cuda")
    AW.AdamW(p).step([g, g])
    assert torch.equal(p[0], p[1]) and p[0][0] != 0


@pytest.mark.parametrize("state", ["f32", "mx8"])
def test_moments_are_copies(state):
    p = torch.zeros(100, device="cuda")
    opt = AW.AdamW([p], state=state)
    opt.step([torch.ones_like(p)])
    for dtype in (torch.float32, torch.bfloat16):
        m, v = opt.moments(dtype)
        kept = m.clone(), v.clone()
        opt.step([torch.full_like(p, 3.0)])
        assert torch.equal(m, kept[0]) and torch.equal(v, kept[1])
        m.zero_(), v.zero_()
        assert opt.m.count_nonzero() >= 100 and opt.v.count_nonzero() >= 100


@pytest.mark.parametrize("state", ["f32", "mx8"])
def test_moments_of_other_tensors_are_refused(state):
    """Equal totals in another order, or another memory order of one tensor."""
    sizes = [64, 128, 32]
    make = lambda s: [torch.ones(n, device="cuda") for n in s]  # noqa: E731
    saved = AW.AdamW(make(sizes), state=state)
    saved.step(make(sizes))
    for other in (make([128, 64, 32]), make([224]), [torch.ones(64, device="cuda"), torch.ones(32, 4, device="cuda").t(),
                                                     torch.ones(32, device="cuda")]):
        opt = AW.AdamW(other, state=state)
        with pytest.raises(ValueError, match="saved"):
            opt.load_state_dict(saved.state_dict())
        assert opt.t == 0 and opt.m.count_nonzero() == 0 and opt.v.count_nonzero() == 0
    f = io.BytesIO()
    torch.save(saved.state_dict(), f)
    f.seek(0)
    opt = AW.AdamW(make(sizes), state=state, seed=4)
    opt.load_state_dict(torch.load(f, weights_only=True))
    assert opt.t == 1 and torch.equal(opt.m, saved.m) and torch.equal(opt.v, saved.v)
    # saved without layouts: sizes are all that is checked
    plain = {k: v for k, v in saved.state_dict().items() if k in ("m", "v", "m_scale", "v_scale", "t", "seed")}
    AW.AdamW(make(sizes), state=state).load_state_dict(plain)


def test_a_refused_state_changes_nothing():
    p = torch.zeros(64, device="cuda")
    opt = AW.AdamW([p])
    sd = {"m": torch.ones(64, device="cuda"), "v": torch.ones(32, device="cuda"), "t": 5, "seed": 1}
    with pytest.raises(ValueError, match="saved"):
        opt.load_state_dict(sd)
    sd = {"m": torch.ones(64, device="cuda"), "v": torch.ones(64, device="cuda"), "seed": 1}
    with pytest.raises((ValueError, KeyError)):
        opt.load_state_dict(sd)
    assert opt.m.count_nonzero() == 0 and opt.t == 0 and opt.seed == 0


def test_layouts_differ_only_where_memory_does():
    """Strides of dimensions of one element say nothing."""
    p = torch.empty_strided((4, 1, 8), (1, 4, 4), device="cuda").zero_()
    g = torch.empty_strided((4, 1, 8), (1, 77, 4), device="cuda").fill_(1.0)
    h = torch.ones(8, 4, device="cuda").t()
    assert not p.is_contiguous() and not g.is_contiguous()
    opt = AW.AdamW([p], weight_decay=0.0, lr=0.5)
    opt.step([g])
    assert torch.all((p + 0.5).abs() < 1e-5)
    opt.step([h])
    with pytest.raises(ValueError, match="differ"):
        opt.step([torch.ones(4, 1, 8, device="cuda")])


@pytest.mark.parametrize("name", ["m", "v"])
def test_moments_at_the_smallest_scales(name):
    """Every code in groups of scales 1 to 40: fp32 is exact (its subnormals
    included), bf16 is the fp32 value rounded to nearest even."""
    opt = AW.AdamW([torch.zeros(40 * 256, device="cuda")], state="mx8")
    codes = torch.arange(256, device="cuda").repeat(40).to(torch.uint8)
    scale = torch.arange(1, 41, device="cuda").repeat_interleave(8).to(torch.uint8)
    getattr(opt, name).copy_(codes)
    getattr(opt, name + "_scale").copy_(scale)
    i = 0 if name == "m" else 1
    want = O.mx8_decode(codes.cpu().numpy(), scale.cpu().numpy(), **(O.M8 if name == "m" else O.V8))
    f32 = opt.moments(torch.float32)[i]
    assert np.array_equal(f32.double().cpu().numpy(), want)
    assert torch.equal(opt.moments(torch.bfloat16)[i], f32.cpu().to(torch.bfloat16).cuda())


def test_bf16_parameters_round_by_the_hash():
    """p rounds up where the hash's 16 bits say so.  fp32 leaves p within tol of
    the exact value, so a code may differ, by one, where a threshold lies within
    tol of it: of n places each with probability 2 tol / spacing at most."""
    n, seed = 50000, 2 ** 33 + 1
    r = np.random.Generator(np.random.PCG64(6))
    p = torch.from_numpy(r.standard_normal(n)).to(torch.bfloat16).cuda()
    opt = AW.AdamW([p], lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, seed=seed)
    p0, m, v = p.double().cpu().numpy(), np.zeros(n), np.zeros(n)
    for step in (1, 2, 3):
        g = torch.from_numpy(r.standard_normal(n) * 0.1).float().cuda()
        opt.step([g])
        g = g.double().cpu().numpy()
        tm = 4 * U * (0.9 * np.abs(m) + 0.1 * np.abs(g)) * 3          # of all steps so far
        p1, m, v = O.adamw(p0, g, m, v, 1e-3, 0.9, 0.95, 1e-8, 0.1, step)
        root = np.sqrt(v / (1 - 0.95 ** step)) + 1e-8
        tol = 1e-3 * (32 * U * np.abs(m) + tm) / (1 - 0.9 ** step) / root + 4 * U * (np.abs(p0) + np.abs(p1))
        bits = ((O.position_hash(np.arange(n), seed, step) * np.uint64(0x5A3C91E7)) & np.uint64(O.MASK)) >> np.uint64(16)
        want = O.round_bf16(p1, bits)
        got = p.double().cpu().numpy()
        spacing = 2.0 ** (np.floor(np.log2(np.abs(p1))) - 7)
        assert np.all(np.abs(got - want) <= spacing * 1.0001)
        few = np.minimum(1.0, 2 * tol / spacing).sum()
        assert (got != want).sum() <= few + 6 * math.sqrt(few) + 6
        p0 = got


def test_bf16_parameters_follow_small_steps_on_average():
    """Steps of 2^-12 below 1, where bf16's spacing is 2^-8: after k of them the
    mean over n entries is 1 - k 2^-12.  A rounding's deviation is at most half a
    spacing, so the mean's is at most 2^-9 sqrt(k / n); fp32 adds k 2^-23."""
    n, k = 1 << 16, 20
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    opt = AW.AdamW([p], lr=2.0 ** -12, betas=(0.9, 0.95), eps=0.0, weight_decay=0.0, seed=11)
    g = torch.ones(n, device="cuda")
    for _ in range(k):
        opt.step([g])
    mean = p.double().mean().item()
    assert abs(mean - (1 - k * 2.0 ** -12)) <= 6 * 2.0 ** -9 * math.sqrt(k / n) + k * 2.0 ** -23
