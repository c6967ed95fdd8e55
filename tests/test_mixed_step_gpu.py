"""The example that runs the operators together: MX4 products forward and
backward, one clipping norm, Shampoo on the matrices, AdamW with 8-bit moments
on the vectors, and single rows through the quantised weights."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_example_trains_and_serves():
    """The loss falls to less than half (an untrained copy of the teacher starts
    at twice the target's variance), and a served row repeats the trained
    network's within fp32's summation order."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import mixed_step
    losses, off = mixed_step.train(steps=40, log=lambda s: print(s, flush=True))
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])
    assert off < 1e-2
