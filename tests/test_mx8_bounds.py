"""How far an MX8 value is from its element (the oracle, whose codes the kernels' equal)."""
import torch

from oracle import layers_oracle as O


def test_the_stated_bounds_hold_and_are_reached():
    """2^-4 of an element whose magnitude is at least 2^-13 of its group's top binade, else 2^-17 of the
    group's largest: E4M3's normal numbers end at 2^-6, 13 binades below [2^7, 2^8), and half a
    step below them is 2^-10."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(4000, 32, generator=gen, dtype=torch.float64) * torch.exp2(-20 * torch.rand(4000, 32, generator=gen))
    x[:, 0] = 128.0
    x[0, 1], x[1, 1], x[2, 1] = 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -6 * (1 + 2.0 ** -4)
    off = (O.mx8_values(x) - x).abs()
    assert (off <= torch.maximum(x.abs() * 2.0 ** -4, torch.full_like(x, 128 * 2.0 ** -17))).all()
    assert off[0, 1] == off[1, 1] == 128 * 2.0 ** -17       # no smaller multiple of the largest bounds it
    normal = x.abs() >= 2.0 ** -6
    assert (off <= x.abs() * 2.0 ** -4)[normal].all()
    assert off[2, 1] == 2.0 ** -10 and x[2, 1] < 2.0 ** -5  # the 13th binade below the top one: half a step


def test_the_documentation_states_them():
    from inverse_root_preconditioning_amd import mx8
    assert "2^-4 of each element, or 2^-17 of the largest of its 32" in mx8.__doc__
