"""Host-side checks of the AdamW, norm and MX4 entry points: struct layouts,
workspace sizes and the synchronous refusal of bad arguments, without a GPU."""
import ctypes

import pytest

from inverse_root_preconditioning_amd import capi as f

FAKE = 0x10000  # a non-null, 16-byte aligned address that is never dereferenced on these paths
NAN, INF = float("nan"), float("inf")


def test_struct_layouts_match_header():
    assert ctypes.sizeof(f.shampoo_tensor) == 24 and f.shampoo_tensor.offset.offset == 16
    assert ctypes.sizeof(f.shampoo_segment) == 8


def _adamw(**kw):
    a = dict(params=FAKE, grads=FAKE, copies=0, hyper=FAKE, ntensors=2, segments=FAKE, nsegments=3, param_dtype=f.T_F32,
             grad_dtype=f.T_F32, state=f.STATE_F32, m=FAKE, v=FAKE, m_scale=0, v_scale=0, lr=1e-3, beta1=0.9, beta2=0.95,
             eps=1e-8, step=1, seed=0, grad_scale=0, stream=0)
    a.update(kw)
    return f.shampoo_adamw(**a)


@pytest.mark.parametrize("bad", [
    dict(params=0), dict(grads=0), dict(hyper=0), dict(segments=0), dict(m=0), dict(v=0), dict(ntensors=-1),
    dict(nsegments=-1), dict(step=0), dict(lr=NAN), dict(lr=INF), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
    dict(beta2=NAN), dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(m=FAKE + 4), dict(v=FAKE + 8),
    dict(m_scale=FAKE), dict(v_scale=FAKE), dict(state=f.STATE_MX8), dict(state=f.STATE_MX8, m_scale=FAKE),
])
def test_adamw_refuses(bad):
    assert _adamw(**bad) == f.EINVAL


@pytest.mark.parametrize("bad", [dict(param_dtype=2), dict(grad_dtype=-1), dict(state=2),
                                 dict(param_dtype=f.T_BF16, copies=FAKE), dict(nsegments=1 << 31)])
def test_adamw_does_not_support(bad):
    assert _adamw(**bad) == f.EUNSUPPORTED


def test_adamw_of_nothing_is_done():
    assert _adamw(ntensors=0, params=0, grads=0, hyper=0, segments=0, nsegments=0, m=0, v=0) == f.OK
    assert _adamw(nsegments=0, m=0, v=0) == f.OK


def test_moments_refusals():
    g = f.shampoo_adamw_moments
    assert g(FAKE, FAKE, FAKE, FAKE, 33, FAKE, FAKE, f.T_F32, 0) == f.EINVAL
    assert g(FAKE, FAKE, FAKE, FAKE, -32, FAKE, FAKE, f.T_F32, 0) == f.EINVAL
    assert g(FAKE, 0, FAKE, FAKE, 32, FAKE, FAKE, f.T_F32, 0) == f.EINVAL
    assert g(FAKE, FAKE, FAKE, FAKE, 32, FAKE, 0, f.T_F32, 0) == f.EINVAL
    assert g(0, 0, 0, 0, 32, 0, 0, f.T_F32, 0) == f.EINVAL
    assert g(FAKE, FAKE, FAKE, FAKE, 32, FAKE, FAKE, 7, 0) == f.EUNSUPPORTED
    assert g(FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE, f.T_F32, 0) == f.OK


def test_norm_refusals_and_workspace():
    g = f.shampoo_grad_norm
    assert g(FAKE, FAKE, -1, f.T_F32, 1.0, FAKE, FAKE, 1 << 20, 0) == f.EINVAL
    for limit in (0.0, -1.0, NAN):
        assert g(FAKE, FAKE, 3, f.T_F32, limit, FAKE, FAKE, 1 << 20, 0) == f.EINVAL
    assert g(FAKE, FAKE, 3, f.T_F32, 1.0, 0, FAKE, 1 << 20, 0) == f.EINVAL
    assert g(0, FAKE, 3, f.T_F32, 1.0, FAKE, FAKE, 1 << 20, 0) == f.EINVAL
    assert g(FAKE, 0, 3, f.T_F32, 1.0, FAKE, FAKE, 1 << 20, 0) == f.EINVAL
    assert g(FAKE, FAKE, 3, 5, 1.0, FAKE, FAKE, 1 << 20, 0) == f.EUNSUPPORTED
    need = f.shampoo_grad_norm_workspace_bytes(100000)
    assert need >= 8 and f.shampoo_grad_norm_workspace_bytes(-1) == 0
    assert g(FAKE, FAKE, 100000, f.T_F32, 1.0, FAKE, FAKE, need - 1, 0) == f.EWORKSPACE
    assert g(FAKE, FAKE, 100000, f.T_F32, 1.0, FAKE, 0, need, 0) == f.EWORKSPACE
    assert g(FAKE, FAKE, 100000, f.T_F32, 1.0, FAKE, FAKE + 4, need, 0) == f.EINVAL


def test_quantize_refusals():
    g = f.shampoo_mx4_quantize
    ok = (FAKE, FAKE, 0, 0, 0)
    assert g(FAKE, 3, 4, 64, 64, *ok) == f.EUNSUPPORTED
    assert g(FAKE, f.T_F32, -1, 64, 64, *ok) == f.EINVAL
    assert g(FAKE, f.T_F32, 4, 64, 63, *ok) == f.EINVAL
    assert g(FAKE, f.T_F32, (1 << 31) + 1, 64, 64, *ok) == f.EUNSUPPORTED
    assert g(0, f.T_F32, 4, 64, 64, *ok) == f.EINVAL
    assert g(FAKE, f.T_F32, 4, 64, 64, 0, 0, 0, 0, 0) == f.EINVAL
    assert g(FAKE, f.T_F32, 4, 64, 64, FAKE, 0, 0, 0, 0) == f.EINVAL
    assert g(FAKE, f.T_F32, 4, 64, 64, FAKE, FAKE, FAKE, 0, 0) == f.EINVAL
    assert g(FAKE, f.T_F32, 4, 64, 64, FAKE + 8, FAKE, 0, 0, 0) == f.EINVAL
    assert g(FAKE, f.T_F32, 4, 64, 64, 0, 0, FAKE, FAKE + 1, 0) == f.EINVAL
    assert g(0, f.T_F32, 0, 64, 64, 0, 0, 0, 0, 0) == f.OK and g(0, f.T_F32, 4, 0, 0, 0, 0, 0, 0, 0) == f.OK
    d = f.shampoo_mx4_dequantize
    assert d(FAKE, FAKE, 4, 64, 0, f.T_F32, 64, 0) == f.EINVAL
    assert d(FAKE, FAKE + 2, 4, 64, FAKE, f.T_F32, 64, 0) == f.EINVAL
    assert d(FAKE, FAKE, 4, 64, FAKE, f.T_F32, 60, 0) == f.EINVAL
    assert d(FAKE, FAKE, 4, 64, FAKE, 9, 64, 0) == f.EUNSUPPORTED
    assert d(0, 0, 0, 64, 0, f.T_F32, 64, 0) == f.OK


def test_product_refusals():
    def g(M=8, N=8, K=64, alpha=1.0, beta=0.0, c=FAKE, dtype=f.T_F32, ldc=8, a=FAKE, bs=FAKE, ws=0, n=0):
        return f.shampoo_mx4_product(a, FAKE, FAKE, bs, M, N, K, alpha, beta, c, dtype, ldc, ws, n, 0)
    assert g(dtype=2) == f.EUNSUPPORTED and g(K=(1 << 24) + 1) == f.EUNSUPPORTED
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(ldc=7), dict(alpha=INF), dict(beta=NAN), dict(c=0), dict(a=0),
                dict(bs=FAKE + 4)):
        assert g(**bad) == f.EINVAL, bad
    assert g(M=0) == f.OK and g(N=0, ldc=0) == f.OK
    # a product whose columns are split needs its workspace
    need = f.shampoo_mx4_workspace_bytes(64, 64, 8192)
    assert need > 0 and f.shampoo_mx4_workspace_bytes(8192, 8192, 8192) == 0
    assert g(M=64, N=64, K=8192, ldc=64) == f.EWORKSPACE
    assert g(M=64, N=64, K=8192, ldc=64, ws=FAKE, n=need - 1) == f.EWORKSPACE
    assert g(M=64, N=64, K=8192, ldc=64, ws=FAKE + 8, n=need) == f.EINVAL
    for bad in ((-1, 4, 4), (4, -1, 4), (4, 4, -1), (1 << 40, 4, 4), (64, 64, 1 << 25)):
        assert f.shampoo_mx4_workspace_bytes(*bad) == 0
        assert f.shampoo_mx4_linear_workspace_bytes(*bad) == 0 or bad[2] == 1 << 25


def test_linear_refusals():
    def g(x=FAKE, ldx=64, w=FAKE, M=100, N=8, K=64, y=FAKE, ldy=8, dtype=f.T_BF16, ws=FAKE, n=1 << 30):
        return f.shampoo_mx4_linear(x, ldx, w, FAKE, M, N, K, y, ldy, dtype, ws, n, 0)
    assert g(dtype=4) == f.EUNSUPPORTED and g(K=(1 << 24) + 1, ldx=1 << 25) == f.EUNSUPPORTED
    for bad in (dict(x=0), dict(ldx=63), dict(w=0), dict(M=-1), dict(y=0), dict(ldy=7), dict(ws=FAKE + 8)):
        assert g(**bad) == f.EINVAL, bad
    assert g(n=16) == f.EWORKSPACE and g(ws=0) == f.EWORKSPACE
    assert g(M=0) == f.OK
    assert f.shampoo_mx4_linear_workspace_bytes(100, 8, 64) >= 100 * 128 // 2
