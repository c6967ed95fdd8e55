"""A tensor that several operations save has one copy in 8 bits, as it has one without."""
import gc

import pytest
import torch

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx8 as M8
from layers_helpers import normal

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
F = torch.nn.functional


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _values(x):
    return M8.dequantize(M8.quantize(x.reshape(-1, x.shape[-1])), x.dtype).view(x.shape)


def test_three_projections_keep_one_copy():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = normal(gen, 4, 64, 256, dtype=BF16).requires_grad_()
    ws = [normal(gen, 8, 256, dtype=BF16).requires_grad_() for _ in range(3)]
    t = x * 1
    torch.autograd.grad(F.linear(x, ws[0]).sum(), (x, ws[0]))   # the library's own workspaces, autograd's thread's too
    gc.collect()
    before = torch.cuda.memory_allocated()
    with M8.saved_tensors():
        ys = [F.linear(t, w) for w in ws]
    held = torch.cuda.memory_allocated() - before - sum(y.numel() * 2 for y in ys)
    assert held <= t.numel() * 33 // 32 + 4 * 512
    dys = [normal(gen, 4, 64, 8, dtype=BF16) for _ in ws]
    got = torch.autograd.grad(ys, ws, dys)
    t8 = _values(t.detach())
    for g, w, dy in zip(got, ws, dys):
        want, = torch.autograd.grad(F.linear(t8, w), w, dy)
        assert torch.equal(g, want)
    # freed with the graph
    del ys, got, g, want
    gc.collect()
    assert torch.cuda.memory_allocated() - before <= sum(d.numel() * 2 for d in dys) + t8.numel() * 2 + 8 * 512


def test_a_change_in_place_makes_another_copy():
    x = torch.randn(64, 64, device="cuda", dtype=BF16).requires_grad_()
    t = x * 1
    with M8.saved_tensors(min_elements=64):
        a = torch.sin(t)
        first = _values(t.detach())
        t.add_(1)
        b = torch.sin(t)
        second = _values(t.detach())
    ga, gb = (torch.autograd.grad(y, x, torch.ones_like(y), retain_graph=True)[0] for y in (a, b))
    assert torch.equal(ga, torch.cos(first)) and torch.equal(gb, torch.cos(second))


def test_parts_and_views_have_their_own():
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = normal(gen, 64, 128, dtype=BF16).requires_grad_()
    t = x * 1
    with M8.saved_tensors(min_elements=64):
        parts = [torch.sin(v) for v in (t, t[:32], t[32:], t.t(), t.view(32, 256), t[:, ::2], t[:32].view(32, 2, 64))]
    for y, v in zip(parts, (t, t[:32], t[32:], t.t(), t.view(32, 256), t[:, ::2], t[:32].view(32, 2, 64))):
        want, = torch.autograd.grad(v, x, torch.cos(_values(v.detach().contiguous())), retain_graph=True)
        assert torch.equal(torch.autograd.grad(y, x, torch.ones_like(y), retain_graph=True)[0], want)


def test_temporaries_at_one_address():
    """Tensors that come and go at the same place are others."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    leaves = [normal(gen, 64, 96, dtype=BF16).requires_grad_() for _ in range(8)]
    with M8.saved_tensors(min_elements=64):
        ys = [torch.sin(x * 1) for x in leaves]
    for x, y in zip(leaves, ys):
        assert torch.equal(torch.autograd.grad(y, x, torch.ones_like(y))[0], torch.cos(_values(x.detach())))


def test_each_stream_has_its_own():
    x = torch.randn(256, 256, device="cuda", dtype=BF16).requires_grad_()
    t = x * 1
    side = torch.cuda.Stream()
    with M8.saved_tensors(min_elements=64):
        a = torch.sin(t)
        side.wait_stream(torch.cuda.current_stream())
        before = torch.cuda.memory_allocated()
        with torch.cuda.stream(side):
            b = torch.sin(t)
    assert torch.cuda.memory_allocated() - before >= t.numel() * 2 + t.numel()
    torch.cuda.current_stream().wait_stream(side)
    want = torch.cos(_values(t.detach()))
    for y in (a, b):
        assert torch.equal(torch.autograd.grad(y, x, torch.ones_like(y), retain_graph=True)[0], want)
    torch.cuda.synchronize()


def test_a_captured_pass_makes_its_own():
    """What is copied during a capture is the graph's: it is made anew by every replay."""
    x = torch.randn(64, 96, device="cuda", dtype=BF16)
    dy = torch.ones_like(x)
    side = torch.cuda.Stream()
    context = M8.saved_tensors(min_elements=64)

    def step(leaf):
        t = leaf * 1
        with context:
            y = torch.sin(t) + torch.sin(t)
        return torch.autograd.grad(y, leaf, dy)[0]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x.clone().requires_grad_())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    static = x.clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static)
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = normal(gen, 64, 96, dtype=BF16)
        static.data.copy_(new)
        want = step(new.clone().requires_grad_())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_one_context_in_several_threads():
    """Threads that save the same tensors at once, each time in other versions."""
    from concurrent.futures import ThreadPoolExecutor
    gen = torch.Generator(device="cuda").manual_seed(4)
    leaves = [normal(gen, 64, 64, dtype=BF16).requires_grad_() for _ in range(3)]
    ts = [x * 1 for x in leaves]
    context = M8.saved_tensors(min_elements=64)
    want = [torch.cos(_values(t.detach())) for t in ts]
    torch.cuda.synchronize()

    def run(i):
        with context:
            for _ in range(20):
                ys = [torch.sin(t) for t in ts] + [torch.sin(t[8 * i:8 * i + 8]) for t in ts]
        got = [torch.autograd.grad(y, t, torch.ones_like(y), retain_graph=True)[0] for y, t in zip(ys, ts)]
        return all(torch.equal(a, b) for a, b in zip(got, want))
    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(run, range(4)))
