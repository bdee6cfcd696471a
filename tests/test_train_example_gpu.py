"""The training example: the loss falls, two runs are equal byte for byte, and 8-bit states follow 32-bit ones."""
import os
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_falls_and_repeats():
    import train_step
    losses, params, states = train_step.train(12, 8)
    again = train_step.train(12, 8)
    assert torch.equal(losses, again[0])
    assert all(torch.equal(a, b) for a, b in zip(params, again[1]))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(states, again[2]))
    assert losses[-1] < losses[0] - 0.5 and torch.isfinite(losses).all()
    full = train_step.train(12, 32)[0]
    assert (full - losses).abs().max() < 0.2
