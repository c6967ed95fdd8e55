"""What the AdamW object keeps, saves and refuses, and the edges of its arithmetic."""
import weakref

import pytest
import torch

from inverse_root_preconditioning_amd import adamw as AW
from inverse_root_preconditioning_amd import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    capi.load()


def test_gradients_are_not_kept_after_the_step():
    p = [torch.zeros(1000, device="cuda"), torch.zeros(50, device="cuda")]
    opt = AW.AdamW(p)
    for as_table in (False, True):
        g = [torch.ones_like(t) for t in p]
        refs = [weakref.ref(t) for t in g]
        if as_table:
            table = AW.TensorTable(g)
            opt.step(table)
            opt.step(table)
            del table
        else:
            opt.step(g)
        del g
        assert all(r() is None for r in refs), as_table


def test_tables_are_checked_after_another_was():
    p = [torch.zeros(64, device="cuda"), torch.zeros(32, device="cuda")]
    opt = AW.AdamW(p)
    opt.step([torch.ones_like(t) for t in p])
    with pytest.raises(ValueError, match="differ from the parameters"):
        opt.step([torch.ones_like(t) for t in reversed(p)])
    opt.step([torch.ones_like(t) for t in p])
    assert opt.t == 2
