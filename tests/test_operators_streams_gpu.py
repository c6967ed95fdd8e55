"""Operands that are freed while a call on another stream has yet to run: their
memory may not be handed out again before it has."""
import pytest
import torch

from inverse_root_preconditioning_amd import adamw as AW
from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import mx4 as MX

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def _like(kind, n=1 << 16):
    """(operands that only the call will hold, call, their memory)."""
    if kind == "grad_norm":
        t = AW.TensorTable([torch.ones(n, device="cuda")])
        return [t], lambda s: AW.grad_norm(t, 1.0, stream=s), [t.tensor, t.segments, *t._keep]
    if kind == "step":
        opt = AW.AdamW([torch.zeros(n, device="cuda")], state="mx8")
        g = torch.ones(n, device="cuda")
        scale = torch.ones(1, device="cuda")
        grads = AW.TensorTable([g])
        mem = [g, scale, opt.m, opt.v, opt.m_scale, opt.v_scale, opt.hyper, opt.params.tensor, grads.tensor,
               grads.segments]
        return [opt, g, scale, grads], lambda s: opt.step(grads, grad_scale=scale, stream=s), mem
    if kind == "moments":
        opt = AW.AdamW([torch.zeros(n, device="cuda")], state="mx8")
        return [opt], lambda s: opt.moments(stream=s), [opt.m, opt.v, opt.m_scale, opt.v_scale]
    x = torch.ones(64, n // 64, device="cuda")
    if kind in ("quantize", "quantize_both"):
        return [x], lambda s: getattr(MX, kind)(x, stream=s), [x]
    q = MX.quantize(x)
    if kind == "dequantize":
        return [q], lambda s: MX.dequantize(q, stream=s), [q._buf]
    if kind == "product":
        other = MX.MX4Matrix(q.codes.clone(), q.scales.clone(), q.rows, q.cols)
        return [q, other], lambda s: MX.product(q, other, stream=s), [q._buf, other.codes, other.scales]
    return [x, q], lambda s: MX.linear(x, q, stream=s), [x, q._buf]


@pytest.mark.parametrize("kind", ["grad_norm", "step", "moments", "quantize", "quantize_both", "dequantize", "product",
                                  "linear"])
def test_memory_in_use_on_another_stream_is_not_handed_out(kind):
    """The stream sleeps before the call.  What is allocated meanwhile, in the
    operands' sizes and without a write, lies elsewhere."""
    stream = torch.cuda.Stream()
    held, call, memory = _like(kind)
    torch.cuda.synchronize()
    places = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in memory}
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)          # some tens of milliseconds
    result = call(stream)
    assert not stream.query()
    del held, call, memory
    fresh = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in places.values() for _ in range(4)]
    assert not {t.data_ptr() for t in fresh} & set(places)
    stream.synchronize()
    del result, fresh
