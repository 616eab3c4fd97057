"""The example trains: the loss starts at ln(vocab) (random weights) and falls, no step overflows."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu


def test_train_block_learns(zopt):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.main(30)
    # rows of unit-variance entries against N(0, 0.02) weights: logits of deviation 0.02 sqrt(256) = 0.32
    assert abs(losses[0] - math.log(m.VOCAB)) < 0.3
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < losses[0] - 2.0  # choosing among the 64 tokens that occur alone is worth ln(64)
