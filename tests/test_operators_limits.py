"""Refusals of the AdamW, norm and MX4 entry points that depend on sizes and
addresses.  Every call here is refused before a launch (no GPU is used)."""
import pytest

from inverse_root_preconditioning_amd import capi as f

FAKE = 0x100000  # a non-null, 16-byte aligned address that is never dereferenced on these paths


@pytest.mark.parametrize("M", [1, 4, 17])
@pytest.mark.parametrize("dtype", [f.T_F32, f.T_BF16])
def test_linear_refuses_an_output_over_its_input(M, dtype):
    """In elements from X: itself, one inside it, one whose end reaches it, rows
    that interleave with its own and share a column."""
    size = 4 if dtype == f.T_F32 else 2

    def g(at, ldx=64, ldy=64, N=64):
        return f.shampoo_mx4_linear(FAKE, ldx, FAKE // 2, FAKE // 2, M, N, 64, FAKE + at * size, ldy, dtype, FAKE // 4,
                                    1 << 20, 0)
    assert g(0) == f.EINVAL
    assert g(63) == f.EINVAL and g((M - 1) * 64 + 63) == f.EINVAL
    assert g(-(M - 1) * 64 - 63) == f.EINVAL
    assert g(63, ldx=200, ldy=200) == f.EINVAL and g(-63, ldx=200, ldy=200) == f.EINVAL
    if M > 1:
        assert g(200 - 63, ldx=200, ldy=200) == f.EINVAL      # reaches the next row
        assert g(64, ldx=200, ldy=100) == f.EINVAL            # rows of another distance within its extent
    assert g(63, ldx=(1 << 63) - 1, ldy=(1 << 63) - 1) == f.EINVAL
