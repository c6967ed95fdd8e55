"""Host-side checks of the entry points of MX8, activations, norms and joins:
struct layouts, workspace sizes and the synchronous refusal of bad arguments.
Every call here is refused, or has nothing to do, before a launch (no GPU is used)."""
import ctypes
import re

import pytest

from inverse_root_preconditioning_amd import build as B
from inverse_root_preconditioning_amd import capi as f

FAKE = 0x10000  # a non-null, 16-byte aligned address that is never dereferenced on these paths
NAN, INF = float("nan"), float("inf")
BIG = (1 << 63) - 1
SIZES = [-(1 << 63), -1, 0, 1, 33, 16384, 16385, 1 << 29, (1 << 29) + 1, 1 << 31, (1 << 31) + 1, BIG]


def test_struct_layouts_match_header():
    """Members of the header's structs, in order, and the packed forms' sizes."""
    text = open(B.ROOT + "/include/shampoo.h").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name in ("shampoo_norm", "shampoo_join", "shampoo_join_grads"):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        members = []
        for line in body.split(";"):
            words = re.findall(r"\w+", line)
            skip = {"const", "void", "int64_t", "double", "uint8_t", "float", "shampoo_norm"}
            members += [w for w in words if w not in skip]
        fields = [n for n, _ in getattr(f, name)._fields_]
        assert members == fields, name
    assert ctypes.sizeof(f.shampoo_norm) == 48
    assert ctypes.sizeof(f.shampoo_join) == f.JOIN.size and ctypes.sizeof(f.shampoo_join_grads) == f.JOIN_GRADS.size
    values = list(range(1, 32))
    for i in (8, 10, 16):
        values[i] = float(values[i])
    packed = f.JOIN.pack(*values)
    j = f.shampoo_join.from_buffer_copy(packed)
    assert (j.rows, j.ld_branch, j.scale, j.after.kind, j.after.eps, j.after.bias_dtype, j.before.eps, j.before.weight,
            j.gate_kind, j.gate_rows, j.before_stats) == (1, 8, 9.0, 10, 11.0, 15, 17.0, 18, 22, 25, 31)


def _sides(rows, cols):
    if rows < 0 or cols < 0:
        return f.EINVAL
    return f.EUNSUPPORTED if rows > 1 << 31 or cols > 1 << 29 else None


def test_every_size_is_refused_with_its_own_code():
    for rows in SIZES:
        for cols in SIZES:
            want = _sides(rows, cols)
            if want is None:
                want = f.OK if rows == 0 or cols == 0 else f.EINVAL
            assert f.shampoo_mx8_quantize(0, f.T_F32, rows, cols, BIG, FAKE, FAKE, 0) == want, (rows, cols)
            assert f.shampoo_mx8_dequantize(FAKE, FAKE, rows, cols, 0, f.T_BF16, BIG, 0) == want, (rows, cols)
            assert f.shampoo_activation(0, FAKE, BIG, 0, 0, rows, cols, f.T_F32, 0, BIG, 0, 0, 0, 0, 0) == want
            assert f.shampoo_activation_backward(0, 0, BIG, FAKE, BIG, 0, 0, 0, 0, 0, 0, 0, rows, cols, f.T_F32, FAKE, BIG,
                                                 0, 0, 0) == want
            if want == f.EINVAL and rows > 0 and cols > f.NORM_COLS:
                want = f.EUNSUPPORTED
            if want == f.OK and cols > f.NORM_COLS:
                want = f.EUNSUPPORTED
            assert _join(rows=rows, cols=cols, residual=0, ld=BIG) == want, (rows, cols)
            need = f.shampoo_join_workspace_bytes(_struct(rows=rows, cols=cols, ld=BIG))
            assert (need > 0) == (0 < rows <= 1 << 31 and 0 < cols <= f.NORM_COLS)


def test_mx8_refusals():
    q, d = f.shampoo_mx8_quantize, f.shampoo_mx8_dequantize
    assert q(FAKE, 2, 4, 64, 64, FAKE, FAKE, 0) == f.EUNSUPPORTED and d(FAKE, FAKE, 4, 64, FAKE, -1, 64, 0) == f.EUNSUPPORTED
    for bad in ((FAKE, 4, 64, 63, FAKE, FAKE), (0, 4, 64, 64, FAKE, FAKE), (FAKE, 4, 64, 64, 0, FAKE),
                (FAKE, 4, 64, 64, FAKE, 0), (FAKE, 4, 64, 64, FAKE + 8, FAKE), (FAKE, 4, 64, 64, FAKE, FAKE + 1)):
        x, rows, cols, ld, codes, scales = bad
        assert q(x, f.T_F32, rows, cols, ld, codes, scales, 0) == f.EINVAL, bad
        assert d(codes, scales, rows, cols, x, f.T_F32, ld, 0) == f.EINVAL, bad
    # 16 rows a workgroup of 2048 (bf16) or 1024 columns
    assert q(FAKE, f.T_BF16, 1 << 31, 1 << 20, 1 << 20, FAKE, FAKE, 0) == f.EUNSUPPORTED
    assert d(FAKE, FAKE, 1 << 31, 1 << 20, FAKE, f.T_F32, 1 << 20, 0) == f.EUNSUPPORTED


def _act(act=0, a=FAKE, lda=64, b=0, ldb=0, rows=4, cols=64, dtype=f.T_F32, y=FAKE, ldy=64, kept=(0, 0, 0, 0)):
    return f.shampoo_activation(act, a, lda, b, ldb, rows, cols, dtype, y, ldy, *kept, 0)


def test_activation_refusals():
    for bad in (dict(act=-1), dict(act=5), dict(dtype=2), dict(rows=1 << 31, cols=1 << 20, lda=BIG, ldy=BIG)):
        assert _act(**bad) == f.EUNSUPPORTED, bad
    for bad in (dict(a=0), dict(lda=63), dict(y=0), dict(ldy=63), dict(b=FAKE, ldb=63), dict(kept=(FAKE, 0, 0, 0)),
                dict(kept=(0, FAKE, 0, 0)), dict(kept=(FAKE + 4, FAKE, 0, 0)), dict(kept=(FAKE, FAKE, FAKE, FAKE)),
                dict(kept=(0, 0, FAKE, FAKE)), dict(b=FAKE, ldb=64, kept=(FAKE, FAKE, 0, 0)),
                dict(b=FAKE, ldb=64, kept=(0, 0, FAKE, FAKE))):
        assert _act(**bad) == f.EINVAL, bad
    assert _act(rows=0, a=0, y=0) == f.OK and _act(cols=0, a=0, y=0) == f.OK

    def back(act=0, dy=FAKE, lddy=64, a=FAKE, lda=64, b=0, ldb=0, kept=(0, 0, 0, 0), gated=0, rows=4, cols=64,
             dtype=f.T_F32, da=FAKE, ldda=64, db=0, lddb=0):
        return f.shampoo_activation_backward(act, dy, lddy, a, lda, b, ldb, *kept, gated, rows, cols, dtype, da, ldda, db,
                                             lddb, 0)
    for bad in (dict(act=9), dict(dtype=7)):
        assert back(**bad) == f.EUNSUPPORTED
    for bad in (dict(dy=0), dict(lddy=63), dict(a=0), dict(lda=63), dict(gated=1), dict(gated=1, b=FAKE, ldb=63),
                dict(db=FAKE, lddb=64), dict(ldda=63), dict(gated=1, b=FAKE, ldb=64, db=FAKE, lddb=63),
                dict(kept=(FAKE, 0, 0, 0)), dict(gated=1, kept=(FAKE, FAKE, 0, 0)), dict(kept=(FAKE + 2, FAKE, 0, 0))):
        assert back(**bad) == f.EINVAL, bad
    assert back(rows=0, dy=0, a=0) == f.OK and back(da=0) == f.OK


def _struct(rows=4, cols=64, stream=f.T_F32, branch=f.T_F32, residual=FAKE, ld=64, y=0, ldy=64, scale=1.0,
            after=(f.NORM_NONE, 0.0, 0, 0, 0, 0), before=(f.NORM_RMS, 1e-6, 0, 0, 0, 0), gate=(f.GATE_NONE, 0, 0, 0),
            kept=(0, 0, 0, 0), stats=(0, 0)):
    return f.JOIN.pack(rows, cols, stream, branch, residual, ld, y, ldy, scale, *after, *before, *gate, *kept, *stats)


def _join(h=FAKE, ldh=None, u=FAKE, ldu=None, **kw):
    ld = kw.get("ld", 64)
    return f.shampoo_join_forward(_struct(**kw), h, ld if ldh is None else ldh, u, ld if ldu is None else ldu, 0)


RMS = (f.NORM_RMS, 1e-6, 0, 0, 0, 0)
NONE = (f.NORM_NONE, 0.0, 0, 0, 0, 0)


@pytest.mark.parametrize("bad", [
    dict(stream=2), dict(branch=-1), dict(stream=f.T_BF16, branch=f.T_F32), dict(before=(3, 1e-6, 0, 0, 0, 0)),
    dict(before=(f.NORM_RMS, 1e-6, FAKE, 4, 0, 0)), dict(before=(f.NORM_RMS, 1e-6, 0, 0, FAKE, 4)), dict(cols=16385, ld=16385),
    dict(y=FAKE, after=(-1, 1e-6, 0, 0, 0, 0)), dict(y=FAKE, gate=(3, FAKE, 0, 0)), dict(y=FAKE, gate=(f.GATE_TOKEN, FAKE, 2, 0)),
])
def test_join_does_not_support(bad):
    assert _join(**bad) == f.EUNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(before=(f.NORM_RMS, 0.0, 0, 0, 0, 0)), dict(before=(f.NORM_RMS, NAN, 0, 0, 0, 0)),
    dict(before=(f.NORM_RMS, INF, 0, 0, 0, 0)), dict(before=(f.NORM_RMS, 1e-60, 0, 0, 0, 0)), dict(before=NONE),
    dict(after=RMS), dict(gate=(f.GATE_ROWS, FAKE, 0, 4)), dict(y=FAKE, gate=(f.GATE_ROWS, FAKE, 0, 3)),
    dict(y=FAKE, gate=(f.GATE_ROWS, FAKE, 0, 0)), dict(y=FAKE, gate=(f.GATE_ROWS, 0, 0, 2)),
    dict(y=FAKE, gate=(f.GATE_TOKEN, 0, 0, 0)), dict(y=FAKE, scale=INF), dict(y=FAKE, scale=1e300), dict(residual=0),
    dict(ld=63, ldh=64, ldu=64), dict(y=FAKE, ldy=63), dict(y=FAKE, h=0), dict(u=0), dict(ldu=63), dict(y=FAKE, ldh=63),
    dict(kept=(FAKE, 0, 0, 0)), dict(kept=(0, FAKE, 0, 0)), dict(kept=(FAKE + 8, FAKE, 0, 0)), dict(kept=(0, 0, FAKE, FAKE)),
    dict(y=FAKE, kept=(0, 0, FAKE, 0)), dict(stats=(0, FAKE + 4)), dict(y=FAKE, after=RMS, stats=(FAKE + 4, FAKE)),
])
def test_join_refuses(bad):
    assert _join(**bad) == f.EINVAL


def test_join_of_nothing_is_done():
    assert _join(rows=0, residual=0, u=0) == f.OK and _join(cols=0, residual=0, u=0) == f.OK
    assert f.shampoo_join_forward(0, FAKE, 64, FAKE, 64, 0) == f.EINVAL
    assert f.shampoo_join_backward(0, 0, FAKE, 1 << 30, 0) == f.EINVAL
    assert f.shampoo_join_backward(_struct(), 0, FAKE, 1 << 30, 0) == f.EINVAL
    assert f.shampoo_join_backward(_struct(rows=0, stats=(0, 0)), f.JOIN_GRADS.pack(*13 * [0]), 0, 0, 0) == f.OK


def _back(dh=0, du=FAKE, dr=FAKE, dy=0, w1=0, b1=0, dgate=0, w2=0, b2=0, lds=(64, 64, 64, 64), ws=FAKE, n=1 << 30, **kw):
    g = f.JOIN_GRADS.pack(dh, lds[0], du, lds[1], dr, lds[2], dy, lds[3], w1, b1, dgate, w2, b2)
    kw.setdefault("stats", (FAKE, FAKE))
    return f.shampoo_join_backward(_struct(**kw), g, ws, n, 0)


@pytest.mark.parametrize("bad", [
    dict(dh=FAKE), dict(dy=FAKE), dict(lds=(64, 63, 64, 64)), dict(lds=(64, 64, 63, 64)), dict(y=FAKE, dh=FAKE, lds=(63, 64, 64, 64)),
    dict(y=FAKE, dy=FAKE, lds=(64, 64, 64, 63)), dict(w1=FAKE), dict(b1=FAKE), dict(dgate=FAKE), dict(w2=FAKE), dict(b2=FAKE),
    dict(du=0), dict(y=FAKE, dh=FAKE, before=NONE), dict(stats=(0, 0)), dict(residual=0), dict(ld=63),
    dict(y=FAKE, after=RMS, stats=(0, FAKE)), dict(y=FAKE, ldy=63), dict(y=FAKE, du=0, dh=FAKE, w2=FAKE,
                                                                       before=(f.NORM_RMS, 1e-6, FAKE, 0, 0, 0)),
    dict(y=FAKE, kept=(FAKE, FAKE, 0, 0)), dict(y=FAKE, kept=(0, 0, FAKE, FAKE)), dict(ws=FAKE + 8),
])
def test_join_backward_refuses(bad):
    assert _back(**bad) == f.EINVAL


def test_join_backward_needs_its_workspace():
    need = f.shampoo_join_workspace_bytes(_struct())
    assert need >= 4 * 64 * 4 // 16
    assert _back(n=need - 1) == f.EWORKSPACE and _back(ws=0, n=need) == f.EWORKSPACE
    size = f.shampoo_join_workspace_bytes
    assert size(0) == 0 and size(_struct(y=FAKE, gate=(f.GATE_ROWS, FAKE, 0, 3))) == 0 and size(_struct(stream=7)) == 0
    # a row of partial sums for every run of rows that shares a row of the gate
    assert size(_struct(rows=1 << 20, y=FAKE, gate=(f.GATE_ROWS, FAKE, 0, 1))) >= (1 << 20) * 64 * 4
    # at most about 768 otherwise
    biased = (f.NORM_LAYER, 1e-6, 0, 0, FAKE, 0)
    for cols in (1, 512, 1000, 4096, 16384):
        for y in (0, FAKE):
            for stream in (f.T_F32, f.T_BF16):
                one = size(_struct(rows=1 << 31, cols=cols, ld=BIG, ldy=BIG, y=y, stream=stream, branch=f.T_BF16, before=biased))
                assert 0 < one <= 4 * 800 * (cols + 8) * 4
