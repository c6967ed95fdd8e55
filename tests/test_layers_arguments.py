"""Arguments of the layers that are checked before any tensor is looked at (no GPU is used)."""
import pytest
import torch

from inverse_root_preconditioning_amd import layers as L

X = torch.zeros(2, 4)


def test_numbers_that_require_a_gradient_are_refused():
    """scale and eps are read as numbers: a gradient of theirs would be dropped without a word."""
    t = torch.tensor(0.5, requires_grad=True)
    with pytest.raises(ValueError, match="scale is a number"):
        L.join(X, X, scale=t)
    with pytest.raises(ValueError, match="eps is a number"):
        L.Norm("rms", eps=t)


def test_texts_are_no_numbers():
    with pytest.raises(TypeError):
        L.join(X, X, scale="0.5")
    with pytest.raises(TypeError):
        L.Norm("rms", eps="1e-6")


def test_other_numbers_are_taken():
    for one in (torch.tensor(0.5), torch.tensor(0.5).numpy(), 1):
        assert L.Norm("rms", eps=one).eps == float(one)
        with pytest.raises(ValueError, match="CUDA tensor"):     # what is wrong here is X
            L.join(X, X, scale=one)
