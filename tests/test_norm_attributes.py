"""A Norm whose attributes are changed is the norm that they say (no GPU is used)."""
import copy
import math
import pickle

import pytest

from inverse_root_preconditioning_amd import capi
from inverse_root_preconditioning_amd import layers as L


def test_a_changed_kind_is_used():
    n = L.Norm("rms", eps=1e-5)
    assert L._parts(n, "n")[:2] == (capi.NORM_RMS, 1e-5)
    n.kind = "layer"
    n.eps = 1e-3
    assert n.kind == "layer" and L._parts(n, "n")[:2] == (capi.NORM_LAYER, 1e-3)
    with pytest.raises(ValueError, match="kind"):
        n.kind = "batch"
    for bad in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(ValueError, match="eps"):
            n.eps = bad
    assert n.kind == "layer" and n.eps == 1e-3


def test_copies():
    n = L.Norm("layer", eps=1e-3)
    for m in (copy.copy(n), copy.deepcopy(n), pickle.loads(pickle.dumps(n))):
        assert L._parts(m, "n") == L._parts(n, "n") and m.kind == "layer"
