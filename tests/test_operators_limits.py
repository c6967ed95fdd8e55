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


BLOCKS = 1 << 24  # the first count of 256-thread workgroups that a launch does not take


def test_adamw_refuses_more_segments_than_a_launch_takes():
    def g(n):
        return f.shampoo_adamw(FAKE, FAKE, 0, FAKE, 1, FAKE, n, f.T_F32, f.T_F32, f.STATE_F32, FAKE, FAKE, 0, 0, 1e-3, 0.9,
                               0.95, 1e-8, 1, 0, 0, 0)
    assert g(BLOCKS) == f.EUNSUPPORTED and g((1 << 31) - 1) == f.EUNSUPPORTED
    n = BLOCKS * 2048                        # 2048 codes a workgroup
    assert f.shampoo_adamw_moments(FAKE, FAKE, FAKE, FAKE, n, FAKE, FAKE, f.T_F32, 0) == f.EUNSUPPORTED


@pytest.mark.parametrize("dtype", [f.T_F32, f.T_BF16])
def test_mx4_refuses_more_workgroups_than_a_launch_takes(dtype):
    """A tall matrix of one column: 64 rows a workgroup along rows, 128 along
    columns, and in dequantisation 64 (bf16) or 32."""
    def quantize(rows, codes, codes_t):
        return f.shampoo_mx4_quantize(FAKE, dtype, rows, 1, 1, codes, codes, codes_t, codes_t, 0)
    assert quantize(64 * BLOCKS, FAKE, 0) == f.EUNSUPPORTED
    assert quantize(128 * BLOCKS, FAKE, FAKE) == f.EUNSUPPORTED and quantize(128 * BLOCKS, 0, FAKE) == f.EUNSUPPORTED
    rows = (64 if dtype == f.T_BF16 else 32) * BLOCKS
    assert f.shampoo_mx4_dequantize(FAKE, FAKE, rows, 1, FAKE, dtype, 1, 0) == f.EUNSUPPORTED


@pytest.mark.parametrize("dtype", [f.T_F32, f.T_BF16])
def test_products_refuse_more_workgroups_than_a_launch_takes(dtype):
    """16 or 32 rows of B a workgroup with few rows of A, else 256 x 256 tiles."""
    def product(M, N):
        return f.shampoo_mx4_product(FAKE, FAKE, FAKE, FAKE, M, N, 64, 1.0, 0.0, FAKE, dtype, N, 0, 0, 0)
    assert product(1, 16 * BLOCKS) == f.EUNSUPPORTED and product(2, 16 * BLOCKS) == f.EUNSUPPORTED
    assert product(16, 32 * BLOCKS) == f.EUNSUPPORTED
    assert product(1 << 31, 512) == f.EUNSUPPORTED
    N = 16 * BLOCKS
    assert f.shampoo_mx4_linear(FAKE, 64, FAKE, FAKE, 1, N, 64, FAKE + (1 << 20), N, dtype, 0, 0, 0) == f.EUNSUPPORTED
