"""Workspace of a join's backward pass: by the gradients that are wanted (host only, nothing is launched)."""
import pytest

from inverse_root_preconditioning_amd import capi as f

FAKE = 0x10000  # a non-null, 16-byte aligned address that is never dereferenced on these paths
NONE = (f.NORM_NONE, 0.0, 0, 0, 0, 0)
RMS = (f.NORM_RMS, 1e-6, FAKE, 0, 0, 0)
BIASED = (f.NORM_LAYER, 1e-6, FAKE, 0, FAKE, 0)
ROWS, COLS = 1 << 16, 64
MATRIX = ROWS * COLS * 4
FEW = 2 * 2 * 800 * (COLS + 8) * 4     # some rows of sums for each of about 768 workgroups


def _struct(after=NONE, before=RMS, run=1):
    gate = (f.GATE_ROWS, FAKE, 0, run) if run else (f.GATE_NONE, 0, 0, 0)
    return f.JOIN.pack(ROWS, COLS, f.T_F32, f.T_F32, FAKE, COLS, FAKE, COLS, 1.0, *after, *before, *gate,
                       0, 0, 0, 0, FAKE, FAKE)


def _grads(w1=0, b1=0, gate=0, w2=0, b2=0):
    return f.JOIN_GRADS.pack(FAKE, COLS, FAKE, COLS, FAKE, COLS, FAKE, COLS, w1, b1, gate, w2, b2)


def _need(join, grads):
    return f.shampoo_join_backward_workspace_bytes(join, grads)


def test_no_sums_over_runs_where_their_gradients_are_not_wanted():
    """A gate of the matrix's own size, and parameters, without gradients: nothing that grows with the rows."""
    for after, before in ((NONE, RMS), (RMS, BIASED), (BIASED, BIASED)):
        join = _struct(after, before)
        assert 0 < _need(join, _grads()) <= FEW
        assert 0 < _need(join, _grads(w2=FAKE)) <= FEW
        assert f.shampoo_join_workspace_bytes(join) >= MATRIX


@pytest.mark.parametrize("after,grads,rows", [
    (NONE, dict(gate=FAKE), 1), (RMS, dict(w1=FAKE), 1), (RMS, dict(w1=FAKE, gate=FAKE), 1), (BIASED, dict(b1=FAKE), 1),
    (BIASED, dict(gate=FAKE), 2), (BIASED, dict(w1=FAKE, b1=FAKE, gate=FAKE), 2)])
def test_a_row_of_sums_for_every_run(after, grads, rows):
    """One for what multiplies the normed branch, another for a bias of its norm; none for the next norm's bias."""
    join = _struct(after, BIASED)
    need = _need(join, _grads(**grads))
    assert rows * MATRIX <= need <= rows * MATRIX + FEW
    assert need <= f.shampoo_join_workspace_bytes(join)
    assert f.shampoo_join_backward(join, _grads(**grads), FAKE, need - 1, 0) == f.EWORKSPACE
    assert f.shampoo_join_backward(join, _grads(**grads), 0, need, 0) == f.EWORKSPACE


def test_without_grads_it_is_enough_for_any():
    for after in (NONE, RMS, BIASED):
        for run in (0, 1, 64, ROWS):
            join = _struct(after, BIASED, run)
            most = f.shampoo_join_workspace_bytes(join)
            assert _need(join, 0) == most
            every = dict(w2=FAKE, b2=FAKE, gate=FAKE if run else 0, w1=FAKE if after is not NONE else 0,
                         b1=FAKE if after is BIASED else 0)
            assert _need(join, _grads(**every)) == most
    assert _need(0, 0) == 0 and _need(_struct(run=3), _grads()) == 0
