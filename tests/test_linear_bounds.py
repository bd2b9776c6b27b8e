"""What the error bounds of tests/linear_bounds.py tell apart (CPU, mistakes planted in the oracle): a state
that lost all but its first 16-bit part, a scale that is off by 1%, a rounding too many."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import linear_bounds as B
from tests import linear_cases as K

SIZES = [(1, 4, 2, 64, 64, 200), (2, 3, 1, 32, 40, 130), (1, 2, 1, 128, 64, 300), (1, 1, 1, 200, 100, 150)]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
def test_the_bound_of_dg_sees_a_lost_part_and_a_scale(name, size):
    a = K.inputs(71, name, *size)
    spans = S.dense_spans(size[0], size[5])
    want, bound = K.backward(a, spans), B.decay_sums(a, name, spans)
    for planted in (dict(x0=K.rounded(a["x0"], "bf16")), dict(dx=K.rounded(a["dx"], "bf16"))):
        assert B.off(K.backward({**a, **planted}, spans)["dg"], want["dg"]) > 2.0 * bound["dg"], planted.keys()
    assert 0.01 * np.linalg.norm(want["dg"]) > 2.0 * bound["dg"] and 0.01 * np.linalg.norm(want["dD"]) > 2.0 * bound["dD"]


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
def test_the_bounds_of_results_see_a_rounding_too_many(name, size):
    """A part as large as the result, rounded before it is added: an operand in one part alone."""
    a = K.inputs(72, name, *size)
    spans = S.dense_spans(size[0], size[5])
    want = {"y": K.forward(a, spans)["y"], **K.backward(a, spans)}
    for n, bound in B.results(a, name, spans).items():
        fine = K.rounded(want[n], name)
        assert B.off(fine, want[n]) < bound, n
        other = np.random.default_rng(73).standard_normal(want[n].shape) * np.abs(want[n])
        assert B.off(K.rounded(want[n] - other, name) + K.rounded(other, name), want[n]) > bound, n
