"""Tolerances and inputs of the tests of the layers."""
import torch

EPS24 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step relative to the value


def check(got, want, magnitude, operations, name="", least=2.0 ** -126):
    """got within its type's rounding of want, `operations` fp32 roundings of
    the terms' magnitude, and `least` (2^-126: below it bf16 and fp32 lose steps)."""
    assert got is not None, name
    want = want.to(got.device)
    got_d = got.double()
    tol = HALF[got.dtype] * want.abs() + (1 + HALF[got.dtype]) * operations * EPS24 * magnitude.to(got.device) + least
    off = (got_d - want).abs()
    bad = ~((off <= tol) | (torch.isnan(want) & torch.isnan(got_d)) | (got_d == want))
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, the first at {bad.nonzero()[0].tolist()}: "
                           f"{got_d[bad][0].item()} for {want[bad][0].item()}, tolerance {tol[bad][0].item()}")


def normal(gen, *shape, dtype=torch.float32, std=1.0, device="cuda"):
    return (torch.randn(*shape, generator=gen, device=device) * std).to(dtype)


def strided(t, kind):
    """t with the same values in another layout: "plain", rows further apart and
    at an odd address, or columns apart."""
    if kind == "plain":
        return t
    lead, cols = t.shape[:-1], t.shape[-1]
    if kind == "padded":
        big = torch.full((*lead, cols + 5), float("nan"), dtype=t.dtype, device=t.device)
        view = big[..., 3:3 + cols]
    else:
        big = torch.full((*lead, cols, 2), float("nan"), dtype=t.dtype, device=t.device)
        view = big[..., 1]
    view.copy_(t)
    return view
