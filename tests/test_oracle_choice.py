"""Pins of the exact choice's oracle: the fp64 oracle where fp64 tells all sums apart, and rows whose order is
known where it does not."""
import numpy as np
import pytest

from oracle import experts as OE
from oracle.choice import choose


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_the_fp64_oracle_where_it_is_exact(kind, biased):
    g = np.random.default_rng(1)
    l, bias = g.normal(size=(15, 24)).astype(np.float32), (0.1 * g.normal(size=24)).astype(np.float32) if biased else None
    for groups, top in ((1, 1), (4, 2), (12, 5)):
        assert np.array_equal(choose(l, 4, kind, bias, groups, top), OE.route_forward(l, 4, kind, bias, groups, top)[0])


def test_sums_that_fp64_does_not_tell_apart():
    l = np.array([[0.0, 40.0, 50.0, 1.0]])
    assert choose(l, 2, "sigmoid", np.zeros(4)).tolist() == [[2, 1]]
    assert choose(l, 2, "sigmoid", np.full(4, 1e10)).tolist() == [[2, 1]]
    assert choose(l, 2, "sigmoid", [0, 1e-30, 0, 0]).tolist() == [[2, 1]]  # e^-40 = 4e-18 is more
    assert choose([[0.0, 80.0, 81.0, 1.0]], 2, "sigmoid", [0, 1e-30, 0, 0]).tolist() == [[1, 2]]  # and e^-80 = 2e-35 less
    assert choose([[0.0, -710.0, -705.0, -720.0]], 4, "softmax", np.zeros(4)).tolist() == [[0, 2, 1, 3]]
    assert choose([[40.0, 41.0, 50.0, 39.0, 42.0, 43.0]], 2, "sigmoid", None, 3, 1).tolist() == [[5, 4]]
    assert choose(np.zeros((1, 4)), 2, "softmax", [0, 0, -3.4e38, 0]).tolist() == [[0, 1]]
