"""The layer, its router's losses and orthogonalised updates together, as the example trains them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_trains(cuda_lib):
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = example.train(steps=40, log=None)
    first, last = history[0], history[-1]
    assert last[0] < 0.8 * first[0]                 # the error against the targets falls
    assert last[3] < first[3]                       # and the busiest expert's share with it
    assert last[1] < first[1]
