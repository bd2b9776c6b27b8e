"""The selective operators' float64 oracle against independent forms: the
convolution against numpy.convolve, the scan against its closed sum, both
gradients against central differences, and packed sequences against separate
ones."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import selective_cases as K


def test_conv_matches_numpy_convolve():
    a = K.conv_inputs(1, "f32", 2, 3, 20, 4, bias=False)
    y, last = S.conv(a["u"], a["w"], None, False, None, S.dense_spans(2, 20))
    for b in range(2):
        for h in range(3):
            assert np.allclose(y[b, h], np.convolve(a["u"][b, h], a["w"][h, ::-1])[:20], atol=1e-12)
    assert np.array_equal(last, a["u"][:, :, -3:])


def test_conv_state_continues_a_sequence():
    a = K.conv_inputs(2, "f32", 1, 3, 20, 4)
    whole, end = S.conv(a["u"], a["w"], a["bias"], True, None, S.dense_spans(1, 20))
    y1, mid = S.conv(a["u"][:, :, :2], a["w"], a["bias"], True, None, S.dense_spans(1, 2))
    y2, end2 = S.conv(a["u"][:, :, 2:], a["w"], a["bias"], True, mid, S.dense_spans(1, 18))
    assert np.allclose(np.concatenate([y1, y2], 2), whole, atol=1e-14) and np.array_equal(end, end2)


def test_scan_matches_the_closed_sum():
    a = K.scan_inputs(3, "f32", 1, 2, 12, 3, gate=False)
    y, last, _ = K.oracle_scan(a, S.dense_spans(1, 12))
    dt = S.softplus(a["delta"] + a["bias"][:, None])[0]
    total = np.cumsum(dt, 1)
    for h in range(2):
        for t in range(12):
            v = a["D"][h] * a["u"][0, h, t]
            for s in range(t + 1):
                decay = np.exp(a["A"][h] * (total[h, t] - total[h, s]))
                v += (a["C"][0, 0, :, t] * decay * a["B"][0, 0, :, s]).sum() * dt[h, s] * a["u"][0, h, s]
            assert abs(v - y[0, h, t]) < 1e-12


def test_packed_sequences_are_separate_ones():
    offs = [2, 7, 7, 8, 15]
    a = K.scan_inputs(4, "f32", 1, 4, 18, 3, G=2, state=True, S_=4)
    y, last, _ = K.oracle_scan(a, S.packed_spans(offs))
    assert np.isnan(y[:, :, :2]).all() and np.isnan(y[:, :, 15:]).all() and np.array_equal(last[1], a["x0"][1])
    for s, (_, b, e) in enumerate(S.packed_spans(offs)):
        if e > b:
            one = {k: (v[..., b:e] if k in ("u", "delta", "z", "B", "C") else v) for k, v in a.items()}
            one["x0"] = a["x0"][s:s + 1]
            y1, l1, _ = K.oracle_scan(one, S.dense_spans(1, e - b))
            assert np.array_equal(y1[0], y[0, :, b:e]) and np.array_equal(l1[0], last[s])


def _differences(f, arrays, grads, names, rng, eps=1e-6):
    for name in names:
        v = arrays[name]
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in v.shape)
            old = v[at]
            v[at] = old + eps
            up = f()
            v[at] = old - eps
            down = f()
            v[at] = old
            want = (up - down) / (2 * eps)
            assert abs(grads[name][at] - want) <= 1e-6 * max(1.0, abs(want)), (name, at, grads[name][at], want)


@pytest.mark.parametrize("gate,skip,bias,soft,state", [(True, True, True, True, True), (False, False, False, True, False),
                                                      (True, False, True, False, True)])
def test_scan_gradients_match_differences(gate, skip, bias, soft, state):
    a = K.scan_inputs(5, "f32", 2, 4, 6, 3, G=2, gate=gate, skip=skip, bias=bias, soft=soft, state=state)
    rng = np.random.default_rng(6)
    dy, dlast = rng.standard_normal(a["u"].shape), rng.standard_normal((2, 4, 3))
    spans = S.dense_spans(2, 6, [6, 4])

    def loss():
        y, last, _ = K.oracle_scan(a, spans)
        return np.nansum(y * dy) + (last * dlast).sum()

    g = K.oracle_scan_grad(a, dy, dlast, spans)
    grads = {"u": g["du"], "delta": g["ddelta"], "A": g["dA"], "B": g["dB"], "C": g["dC"], "D": g["dD"],
             "bias": g["ddelta_bias"], "x0": g["dx0"], "z": g.get("dz")}
    grads = {k: None if v is None else np.nan_to_num(v) for k, v in grads.items()}
    _differences(loss, a, grads, [k for k in grads if a[k] is not None], rng)


@pytest.mark.parametrize("W,act,state", [(4, True, True), (3, False, False), (1, True, False), (2, True, True)])
def test_conv_gradients_match_differences(W, act, state):
    a = K.conv_inputs(7, "f32", 2, 3, 5, W, state=state)
    rng = np.random.default_rng(8)
    dy, dlast = rng.standard_normal(a["u"].shape), rng.standard_normal((2, 3, W - 1))
    spans = S.dense_spans(2, 5, [5, 1])

    def loss():
        y, last = S.conv(a["u"], a["w"], a["bias"], act, a["state"], spans)
        return np.nansum(y * dy) + (last * dlast).sum()

    g = S.conv_grad(a["u"], a["w"], a["bias"], act, a["state"], dy, dlast, spans)
    grads = {"u": np.nan_to_num(g["du"]), "w": g["dweight"], "bias": g["dbias"], "state": g["dstate"]}
    _differences(loss, a, grads, [k for k in grads if a[k] is not None], rng)
