"""Pins of the float64 oracle of the AdamW step and the MX4 matrices, by closed
forms and independent implementations (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import adamw_mx4_oracle as O


def _rng(key):
    return np.random.Generator(np.random.PCG64(key))


@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_adamw_steps_equal_torch_float64(decay):
    r = _rng(1)
    p = torch.tensor(r.standard_normal(50), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=decay)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 5):
        g = r.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        q, m, v = O.adamw(q, g, m, v, 1e-2, 0.9, 0.95, 1e-8, decay, t)
        assert np.abs(q - p.detach().numpy()).max() < 1e-13


def test_mx8_m_codes_are_ocp_e4m3():
    code = np.arange(256, dtype=np.uint8)
    keep = (code & 127) != 127            # NaN in the OCP table, never written by the encoder
    ours = O.mx8_decode(code, np.full(8, 127), **O.M8)
    theirs = torch.from_numpy(code).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours[keep], theirs[keep])


def test_mx8_v_codes_are_three_mantissa_bits_below_the_exponent():
    v = O.mx8_decode(np.arange(256), np.full(8, 127), **O.V8)
    assert v[0] == 0 and v[1] == 2.0 ** -17 and v[8] == 2.0 ** -14 and v[255] == 1.875 * 2.0 ** 16
    assert np.all(np.diff(v) > 0)


@pytest.mark.parametrize("fmt", [O.M8, O.V8])
def test_mx8_round_trip_is_exact_on_its_own_values(fmt):
    r = _rng(2)
    code = r.integers(8, 8 * (fmt["back"] + fmt["bias"] + 1), 320)     # normal codes, the top of each group's range last
    code[31::32] = 8 * (fmt["back"] + fmt["bias"]) + 3
    scale = r.integers(60, 180, 10)
    x = O.mx8_decode(code, scale, **fmt)
    for h in (0, 65535):
        c, s = O.mx8_encode(x, np.full(320, h), **fmt)
        assert np.array_equal(s, scale) and np.array_equal(c, code)


@pytest.mark.parametrize("fmt", [O.M8, O.V8])
def test_mx8_rounds_to_either_neighbour_with_the_right_mean(fmt):
    x = np.concatenate([[1.0], _rng(3).uniform(2.0 ** -6, 1.0, 31)])
    low = O.mx8_decode(*O.mx8_encode(x, np.zeros(32), **fmt), **fmt)
    h = np.arange(0, 65536, 64)
    got = np.stack([O.mx8_decode(*O.mx8_encode(x, np.full(32, k), **fmt), **fmt) for k in h])
    assert np.all(got.min(0) <= x + 1e-12) and np.all(got.max(0) >= x - 1e-12)
    assert np.all(got.max(0) - got.min(0) <= x / 8 * (1 + 1e-9))         # neighbours are at most an eighth apart
    assert np.abs(got.mean(0) - x).max() <= 2.0 / len(h) / 8             # the grid of hashes resolves 1 / len(h) of a spacing
    assert np.all(low <= x + 1e-12)


def test_mx8_special_groups():
    x = np.zeros(96)
    x[32], x[40] = np.nan, 3.0
    x[64] = 1.0
    c, s = O.mx8_encode(x, np.full(96, 7), **O.V8)
    assert list(s) == [1, 255, 112] and np.all(c[:32] == 1) and np.all(c[32:64] == 0)
    assert np.all(np.isnan(O.mx8_decode(c, s, **O.V8)[32:64]))
    c, s = O.mx8_encode(x, np.full(96, 7), **O.M8)
    assert list(s) == [1, 255, 120] and np.all(c[:32] == 0)


def test_mx4_values_ties_and_saturation():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, 0.2501, -0.75, -5.0, 6.0, 4.0]])
    want = np.array([[0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 0.5, -1.0, -4.0, 6.0, 4.0]])
    code, s = O.mx4_quantize(x)
    assert s[0, 0] == 127
    assert np.array_equal(O.mx4_values(code, s, 13), want)
    assert np.array_equal(O.mx4_round(x * 2.0 ** 40), want * 2.0 ** 40)


def test_mx4_zero_nan_and_tiny_groups():
    x = np.zeros((1, 128))
    x[0, 33], x[0, 64], x[0, 96] = np.inf, 2.0 ** -130, 2.0 ** -126
    code, s = O.mx4_quantize(x)
    assert list(s[0]) == [0, 255, 0, 0]
    v = O.mx4_values(code, s, 128)
    assert v[0, 0] == 0 and np.all(np.isnan(v[0, 32:64])) and v[0, 96] == 2.0 ** -126
    assert v[0, 64] == 0                                                 # 2^-3 of the smallest scale


def test_mx4_relative_error_is_within_half_a_spacing():
    x = _rng(4).standard_normal((16, 320))
    q = O.mx4_round(x)
    top = np.abs(x.reshape(16, -1, 32)).max(2)
    scale = 2.0 ** (np.floor(np.log2(top)) - 2)
    # spacing 2 at most below 6; from 6 up to 8 the value saturates
    assert np.all(np.abs(q - x).reshape(16, -1, 32) <= 2.0 * scale[..., None])


def test_position_hash_halves_are_uniform_and_differ_by_step():
    h = O.position_hash(np.arange(1 << 18), 5, 3)
    for half in (h & np.uint64(0xFFFF), h >> np.uint64(16)):
        u = half.astype(np.float64) / 65536
        assert abs(u.mean() - 0.5) < 5 / math.sqrt(12 * u.size)
    other = O.position_hash(np.arange(1 << 18), 5, 4)
    assert abs(np.corrcoef(h.astype(float), other.astype(float))[0, 1]) < 5 / 512
    big = O.position_hash(np.array([5, 5 + (1 << 32)]), 1, 1)
    assert big[0] != big[1]


def test_bf16_rounds_to_either_neighbour_with_the_right_mean():
    x = np.concatenate([_rng(5).standard_normal(60), [1.0, -1.5, 2.0 ** -127, 0.0]])
    x = x.astype(np.float32).astype(np.float64)
    up = np.stack([O.round_bf16(x, np.full(64, h)) for h in range(0, 65536, 64)])
    for row in (up[0], up[-1]):
        assert np.array_equal(torch.from_numpy(row).to(torch.bfloat16).double().numpy(), row)
    spacing = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 7)
    assert np.all(np.abs(up - x) < spacing) and np.all(np.abs(up.mean(0) - x) <= spacing / 1024)
    assert np.all(up[:, 60:] == x[60:])                                  # bf16's own values stay


def test_a_moment_that_vanishes_beside_its_group_keeps_a_root():
    """Code 1 stands for at least 2^-33 of the group's largest v, 2^-16.5 of its root."""
    worst = 1.0
    for top in (1.0, 1.5, 1.99999):
        x = np.zeros(32)
        x[3] = top
        v = O.mx8_decode(*O.mx8_encode(x, np.zeros(32), **O.V8), **O.V8)
        worst = min(worst, math.sqrt(v[0] / top))
    assert 2.0 ** -16.5 <= worst < 2.0 ** -16.49
