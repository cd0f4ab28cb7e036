"""examples/distill_head.py: both losses fall when a student is trained on them
through the library's forward and backward calls."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_distill_head_example_learns():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_head.py")
    spec = importlib.util.spec_from_file_location("distill_head", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=40)
    first, last = losses[0], losses[-1]
    # an untrained head is near uniform: log 4099 = 8.3
    assert 7.5 < first[0] < 9.5
    assert last[0] < 0.7 * first[0] and last[1] < 0.7 * first[1]
