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


SIZES = [-(1 << 63), -1, 0, 1, 16, 17, 64, 127, 128, 129, 8192, 1 << 24, (1 << 24) + 1, 1 << 31, (1 << 31) + 1,
         (1 << 63) - 1]


def _sides(*sizes):
    """The code that the sizes alone decide, else None."""
    if min(sizes) < 0:
        return f.EINVAL
    return f.EUNSUPPORTED if max(sizes) > 1 << 31 else None


def test_every_size_is_refused_with_its_own_code():
    """Without an output (or an input) every call ends before a launch: negative
    sizes, then sizes beyond the limits, then empty results, then the pointer."""
    big = (1 << 63) - 1
    for m in SIZES:
        for n in SIZES:
            for k in SIZES:
                want = _sides(m, n, k)
                if want is None:
                    want = f.EUNSUPPORTED if k > 1 << 24 else f.OK if m == 0 or n == 0 else f.EINVAL
                assert f.shampoo_mx4_product(FAKE, FAKE, FAKE, FAKE, m, n, k, 1.0, 0.0, 0, f.T_F32, big, 0, 0, 0) == want
                assert f.shampoo_mx4_linear(FAKE, big, FAKE, FAKE, m, n, k, 0, big, f.T_F32, 0, 0, 0) == want, (m, n, k)
            want = _sides(m, n)
            if want is None:
                want = f.OK if m == 0 or n == 0 else f.EINVAL
            assert f.shampoo_mx4_quantize(0, f.T_F32, m, n, big, FAKE, FAKE, 0, 0, 0) == want, (m, n)
            assert f.shampoo_mx4_dequantize(FAKE, FAKE, m, n, 0, f.T_BF16, big, 0) == want, (m, n)
        want = f.OK if m == 0 else f.EINVAL
        assert f.shampoo_adamw(FAKE, FAKE, 0, FAKE, 1, FAKE, m, f.T_F32, f.T_F32, f.STATE_F32, 0, FAKE, 0, 0, 1e-3, 0.9,
                               0.95, 1e-8, 1, 0, 0, 0) == want, m
        want = f.EINVAL if m < 0 or m % 32 or m else f.OK
        assert f.shampoo_adamw_moments(0, 0, 0, 0, m, 0, 0, f.T_F32, 0) == want, m
