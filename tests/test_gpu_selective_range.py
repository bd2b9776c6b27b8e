"""The selective scan where steps, decays and inputs leave the ordinary range:
negative steps, decays beyond float32 over zero states, infinite inputs.  Same
oracle and tolerances as tests/test_gpu_selective.py."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import selective_cases as K
from tests.test_gpu_selective import _check_scan, _check_scan_backward

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _plain_inputs(seed, Bsz, H, L, N, G=1, **kw):
    """float32 inputs whose delta is dt itself: no softplus, no bias."""
    return K.scan_inputs(seed, "f32", Bsz, H, L, N, G, gate=True, soft=False, bias=False, state=True, **kw)


@pytest.mark.parametrize("order", ["rows", "tokens", "mixed"])
@pytest.mark.parametrize("L", [40, 700])   # one chunk; chunks of 64 steps
@pytest.mark.parametrize("N", [1, 3, 8, 16, 20, 40])
def test_negative_steps(order, N, L):
    # a chunk's steps add up to about -192, one step alone is -200; |dt A| < 1, so that
    # every state, and every gradient, stays ordinary
    a = _plain_inputs(61, 1, 5, L, N)
    r = np.random.default_rng(62)
    a["delta"] = K.rounded(-3.0 * np.exp(0.1 * r.standard_normal(a["delta"].shape)), "f32")
    a["delta"][0, :, 17] = -200.0
    a["A"] = K.rounded(-1e-3 * (1.0 + np.arange(N)) / N * np.exp(0.1 * r.standard_normal((5, N))), "f32")
    _check_scan(a, "f32", order, S.dense_spans(1, L))
    _check_scan_backward(a, "f32", order, S.dense_spans(1, L))
