"""How near linear attention's results are to the definition, where elementwise bounds on
sums of magnitudes would let a systematic rounding pass."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import linear_bounds as B
from tests import linear_cases as K
from tests.test_gpu_linear import DEV, _f32, _np, _ssm, check

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


def within_bounds(a, name, order="tokens", offsets=None):
    ssm = _ssm()
    Bsz, _, _, L = a["v"].shape
    spans = S.dense_spans(Bsz, L) if offsets is None else S.packed_spans(offsets)
    args, kw = K.call_args(a, name, order)
    if offsets is not None:
        kw["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    f = ssm.linear_attention(*args, **kw, want_state=True, save=True)
    g = ssm.linear_attention_backward(*args, K.on_device(a["dy"], name, order), dx=_f32(a["dx"]), saved=f["saved"], **kw)
    want = {"y": K.forward(a, spans)["y"], **K.backward(a, spans)}
    bounds = B.decay_sums(a, name, spans)
    if name != "f32":
        bounds.update(B.results(a, name, spans))
    got = {"y": f["y"], **g}
    off = {n: B.off(_np(got[n]), want[n]) / bounds[n] for n in bounds if got.get(n) is not None}
    assert max(off.values()) <= 1.0, off


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", [(1, 4, 2, 64, 64, 200), (2, 3, 1, 32, 40, 130), (1, 2, 1, 128, 64, 300), (1, 1, 1, 200, 100, 150),
                                  (1, 36, 1, 64, 64, 100)])
def test_errors_are_those_of_independent_roundings(name, size):
    within_bounds(K.inputs(71, name, *size), name)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_errors_without_what_is_optional_and_in_packed_rows(name):
    within_bounds(K.inputs(72, name, 2, 2, 1, 48, 64, 140, beta=False, skip=False, carry=False), name, "rows")
    within_bounds(K.inputs(73, name, 1, 2, 2, 64, 32, 260, S=4), name, "tokens", [0, 1, 66, 194, 260])


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [64, 256])
def test_many_pieces(name, N):
    """A sequence in more pieces than are read at once: ten of the fewest steps (four chunks), in either direction, on
    states that reach through all of them."""
    L = 10 * 4 * B.chunk(name) + 5
    a = K.inputs(74, name, 1, 1, 1, N, 24, L, pace=2e-3)
    ssm = _ssm()
    pieces = ssm.linear_bytes(ssm.OP_LINEAR_ATTENTION, K.torch_type(name), 1, 1, N, 24, 1, L) // (N * 24 * 4)
    assert pieces >= 11
    check(a, name, "tokens")
    within_bounds(a, name)
    b = K.inputs(75, name, 1, 1, 1, N, 24, L, S=2, pace=2e-3)
    check(b, name, "tokens", offsets=[3, 100, L - 1])
