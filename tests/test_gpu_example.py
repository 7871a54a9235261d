"""examples/train_step.py: the operators together, as a training loop uses them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_the_layer_learns():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, load = m.train(steps=40, T=1024)
    assert all(v == v and v < 1e3 for v in losses)
    assert sum(losses[-5:]) / 5 < 0.8 * losses[0]
    assert max(load[-5:]) < 16 / 4 / 2  # (all tokens on the same experts would be 16 / 4)
