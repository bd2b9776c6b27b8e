"""How near linear attention's results are to the definition, where elementwise bounds on
sums of magnitudes would let a systematic rounding pass."""
import numpy as np
import pytest

from tests import linear_cases as K
from tests.test_gpu_linear import _f32, _np, _ssm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["tokens", "rows", "mixed"])
@pytest.mark.parametrize("size", [(1, 6, 2, 32, 64, 130), (2, 2, 1, 100, 37, 70), (1, 1, 1, 16, 24, 900)])
def test_the_skip_is_rounded_once(name, order, size):
    """Where the states are zero y is D v and dv is D dy: a product in float32 (2^-24), rounded to the type."""
    ssm = _ssm()
    a = K.inputs(51, name, *size, carry=False)
    a["k"] = np.zeros_like(a["k"])
    a["D"] = K.rounded(1.0 + np.random.default_rng(52).random(size[1]), "f32")
    args, kw = K.call_args(a, name, order)
    y = _np(ssm.linear_attention(*args, **kw)["y"])
    a["k"], a["q"] = K.rounded(np.random.default_rng(53).standard_normal(a["k"].shape), name), np.zeros_like(a["q"])
    args, kw = K.call_args(a, name, order)
    dv = _np(ssm.linear_attention_backward(*args, K.on_device(a["dy"], name, order), **kw)["dv"])
    for got, v in ((y, a["v"]), (dv, a["dy"])):
        want = a["D"][:, None, None] * v
        half = K.HALF_STEP[name] if name != "f32" else 0.0
        assert (np.abs(got - want) <= np.abs(want) * (half * (1.0 + 2.0 * K.U) + 2.0 * K.U) + K.SMALLEST[name]).all()
