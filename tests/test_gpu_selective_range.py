"""The selective scan where steps, decays and inputs leave the ordinary range:
negative steps, decays beyond float32 over zero states, infinite inputs.  Same
oracle and tolerances as tests/test_gpu_selective.py."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import selective_cases as K
from tests.test_gpu_selective import DEV, _check_scan, _check_scan_backward, _f32, _np, _scan_args, _ssm

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


# Growing states (dt A > 0): over a chunk of 64 steps they grow by e^96, more than
# float32 holds, while every state and gradient stays in its range.

@pytest.mark.parametrize("order", ["rows", "tokens", "mixed"])
@pytest.mark.parametrize("N", [1, 16, 20, 40])
def test_zero_states_through_growing_chunks(order, N):
    # inputs in the last 20 of 700 steps only: the states before them are zero
    a = _plain_inputs(63, 1, 5, 700, N)
    a["delta"][...], a["A"][...], a["x0"][...] = 0.125, 12.0, 0.0
    a["u"][..., :680] = 0.0
    _check_scan(a, "f32", order, S.dense_spans(1, 700))
    # from the end: C in the first 20 steps only, and no input at all
    a["u"][...] = 0.0
    a["C"][..., 20:] = 0.0
    _check_scan_backward(a, "f32", order, S.dense_spans(1, 700), dlast=False)


@pytest.mark.parametrize("order", ["rows", "tokens", "mixed"])
@pytest.mark.parametrize("N", [1, 16, 20, 40])
def test_small_states_through_a_growing_chunk(order, N):
    # states of 2^-80 (e^-55) that grow by e^96 in the second chunk and shrink by e^-78
    # in the third; gradients go through the same from the end
    a = _plain_inputs(64, 1, 5, 180, N)
    a["A"][...], a["u"][...] = 12.0, 0.0
    a["delta"][..., :64], a["delta"][..., 64:128], a["delta"][..., 128:] = 2.0 ** -13, 0.125, -0.125
    a["x0"] = K.rounded(a["x0"] * 2.0 ** -80, "f32")
    a["C"][..., 64:] = 0.0
    _check_scan(a, "f32", order, S.dense_spans(1, 180))
    _check_scan_backward(a, "f32", order, S.dense_spans(1, 180))


def _assert_like_definition(got, want, mag, name, roundings, what):
    """Infinities where the definition has them, with their signs; near it elsewhere."""
    inf = np.isinf(want)
    assert not np.isnan(want).any() and np.array_equal(got[inf], want[inf]), what
    K.assert_near(np.where(inf, 0.0, got), np.where(inf, 0.0, want), np.where(inf, 0.0, mag), name, roundings, what)


def _infinite_inputs(name, Bsz, L, N, at, value):
    # all of one sign but u's and the gate's: every infinite sum has a sign
    a = K.scan_inputs(65, name, Bsz, 5, L, N, gate=True, state=True)
    for k in ("B", "C", "D"):
        a[k] = np.abs(a[k]) + 0.5
    a = {k: K.rounded(v, name) if k in ("B", "C") else K.rounded(v, "f32") if k == "D" else v for k, v in a.items()}
    a["u"][0, 1, at], a["u"][0, 3, at] = value, -value
    return a


@pytest.mark.parametrize("name,order", [("f32", "rows"), ("bf16", "tokens"), ("f32", "mixed")])
@pytest.mark.parametrize("L,at", [(40, 3), (40, 33), (200, 70), (200, 199)])
@pytest.mark.parametrize("N", [1, 2, 3, 8, 16, 20, 33, 40])
def test_infinite_inputs(name, order, L, at, N):
    # an infinite u makes its channel's states and outputs infinite from its step on,
    # however the state count fills the lanes, and leaves the other channels alone
    a = _infinite_inputs(name, 1, L, N, at, np.inf)
    args, more = _scan_args(a, name, order)
    out = _ssm().selective_scan(*args, **more, want_state=True)
    want, last, _ = K.oracle_scan(a, S.dense_spans(1, L))
    mag, mlast, _ = K.oracle_scan(a, S.dense_spans(1, L), mag=True)
    assert np.isinf(want).sum() == 2 * (L - at)
    _assert_like_definition(_np(out["y"]), want, mag, name, K.steps_bound(L, N), "y")
    _assert_like_definition(_np(out["x"]), last, mlast, "f32", K.steps_bound(L, N), "x")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 3, 8, 16, 20, 33, 40])
def test_infinite_token(name, N):
    a = _infinite_inputs(name, 2, 1, N, 0, np.inf)
    tok = lambda v: torch.from_numpy(v[..., 0]).to(K.torch_type(name)).to(DEV)  # noqa: E731
    x = _f32(a["x0"])
    y = _ssm().selective_step(tok(a["u"]), tok(a["delta"]), _f32(a["A"]), tok(a["B"]), tok(a["C"]), x, D=_f32(a["D"]),
                              z=tok(a["z"]), delta_bias=_f32(a["bias"]), softplus=True)["y"]
    want, last, _ = K.oracle_scan(a, S.dense_spans(2, 1))
    mag, mlast, _ = K.oracle_scan(a, S.dense_spans(2, 1), mag=True)
    _assert_like_definition(_np(y), want[..., 0], mag[..., 0], name, K.steps_bound(1, N), "y")
    _assert_like_definition(_np(x), last, mlast, "f32", K.steps_bound(1, N), "x")


@pytest.mark.parametrize("name,order", [("f32", "rows"), ("bf16", "tokens"), ("f32", "mixed")])
@pytest.mark.parametrize("L,at", [(40, 3), (200, 70)])
@pytest.mark.parametrize("N", [1, 3, 8, 16, 20, 40])
def test_gradients_beside_infinite_inputs(name, order, L, at, N):
    # an infinite u leaves the gradients of the other channels as they are, bit for bit,
    # and its own channel's du, which holds no u
    grads = []
    for value in (1.0, np.inf):
        a = _infinite_inputs(name, 1, L, N, at, value)
        args, more = _scan_args(a, name, order)
        dy = K.on_device(K.rounded(np.random.default_rng(66).standard_normal(a["u"].shape), name), name, order)
        f = _ssm().selective_scan(*args, **more, save=True)
        grads.append(_ssm().selective_scan_backward(*args, dy, **more, saved=f["saved"]))
    others = [0, 2, 4]
    for k in ("ddelta", "dz", "dx0"):
        assert torch.equal(grads[0][k][:, others], grads[1][k][:, others]), k
    for k in ("dA", "dD", "ddelta_bias"):
        assert torch.equal(grads[0][k][others], grads[1][k][others]), k
    assert torch.equal(grads[0]["du"], grads[1]["du"])
    assert bool(torch.isfinite(grads[0]["du"]).all())
