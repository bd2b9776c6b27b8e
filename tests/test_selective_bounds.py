"""The bounds of tests/selective_bounds.py hold for a float32 evaluation of the scan
on the CPU, and mistakes that coarser tolerances let pass go beyond them."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import selective_bounds as T
from tests import selective_cases as K

CASES = [(2, 6, 300, 16, 2), (1, 3, 900, 5, 1)]


def _float32(a, dy, dlast, state=np.float32, decay=1.0):
    """The scan and its gradients step by step in numpy's float32; `state` holds the states."""
    f = np.float32
    a = {k: w.astype(f) if isinstance(w, np.ndarray) else w for k, w in a.items()}
    n, H, L = a["u"].shape
    N, G = a["A"].shape[1], a["B"].shape[1]
    rep = H // G
    v = a["delta"] + a["bias"][:, None]
    dt, sig = np.logaddexp(v, f(0)), f(1) / (f(1) + np.exp(-a["z"]))
    gate = a["z"] * sig
    wide = lambda w, t: np.repeat(w[:, :, :, t], rep, 1)  # noqa: E731
    x, xs, decs, pre = a["x0"].astype(state).astype(f), [], [], np.zeros_like(v)
    xs.append(x)
    for t in range(L):
        dec = np.exp(dt[:, :, t, None] * a["A"]) * f(decay if t == L // 2 else 1.0)
        x = (dec * x + (dt * a["u"])[:, :, t, None] * wide(a["B"], t)).astype(state).astype(f)
        pre[:, :, t] = (wide(a["C"], t) * x).sum(2, dtype=f) + a["D"] * a["u"][:, :, t]
        xs.append(x), decs.append(dec)
    out = dict(y=pre * gate, x=x)
    dy = dy.astype(f)
    p = dy * gate
    out["dz"] = dy * sig * (f(1) + a["z"] * (f(1) - sig)) * pre
    carry, slope = dlast.astype(f), f(1) / (f(1) + np.exp(-v))
    out.update(du=np.zeros_like(v), ddelta=np.zeros_like(v), dB=np.zeros_like(a["B"]), dC=np.zeros_like(a["C"]),
               dA=np.zeros((H, N), f))
    for t in range(L - 1, -1, -1):
        g = carry + p[:, :, t, None] * wide(a["C"], t)
        sums = lambda w: w.reshape(n, G, rep, N).sum(2, dtype=f)  # noqa: E731
        out["dB"][..., t] = sums(g * (dt * a["u"])[:, :, t, None])
        out["dC"][..., t] = sums(p[:, :, t, None] * xs[t + 1])
        gB = (g * wide(a["B"], t)).sum(2, dtype=f)
        carry = decs[t] * g
        back = carry * xs[t]
        out["dA"] += (back * dt[:, :, t, None]).sum(0, dtype=f)
        out["du"][:, :, t] = a["D"] * p[:, :, t] + dt[:, :, t] * gB
        out["ddelta"][:, :, t] = slope[:, :, t] * (a["u"][:, :, t] * gB + (back * a["A"]).sum(2, dtype=f))
    out.update(dx0=carry, dD=(p * a["u"]).sum((0, 2), dtype=np.float64), ddelta_bias=out["ddelta"].sum((0, 2), dtype=np.float64))
    return out


def _setting(case, seed):
    Bsz, H, L, N, G = case
    a = K.scan_inputs(seed, "f32", Bsz, H, L, N, G, state=True)
    r = np.random.default_rng(seed + 1)
    dy = K.rounded(r.standard_normal((Bsz, H, L)), "f32")
    dlast = K.rounded(r.standard_normal((Bsz, H, N)), "f32")
    spans = S.dense_spans(Bsz, L)
    y, last, _ = K.oracle_scan(a, spans)
    want = dict(y=y, x=last, **K.oracle_scan_grad(a, dy, dlast, spans))
    return a, dy, dlast, want, T.scan_bounds(a, spans, dy, dlast)


@pytest.mark.parametrize("case", CASES)
def test_bounds_hold_and_are_tight(case):
    a, dy, dlast, want, err = _setting(case, 81)
    got = _float32(a, dy, dlast)
    for k in got:
        T.within(got[k], want[k], err[k], "f32", k)
    # they do not grow with the sequence's length as a count of its steps does (300 steps: 6e-4, 900: 1.7e-3)
    for k in ("y", "du"):
        assert np.median(err[k]) <= 1e-4 * np.median(np.abs(want[k])), k


# states held in float16; one step's decay off by 0.2%
@pytest.mark.parametrize("mistake", [dict(state=np.float16), dict(decay=1.0 + 2e-3)])
@pytest.mark.parametrize("case", CASES)
def test_mistakes_go_beyond_them(case, mistake):
    a, dy, dlast, want, err = _setting(case, 82)
    got = _float32(a, dy, dlast, **mistake)
    for k in ("y", "x", "dC", "dz", "ddelta") if "state" in mistake else ("y", "du", "dB", "dC"):
        with pytest.raises(AssertionError):
            T.within(got[k], want[k], err[k], "f32", k)


def test_packed_bounds_are_the_sequences():
    a = K.scan_inputs(83, "f32", 1, 4, 60, 8, 2, state=True, S_=3)
    dy = K.rounded(np.random.default_rng(84).standard_normal((1, 4, 60)), "f32")
    spans = S.packed_spans([5, 25, 25, 50])
    got = T.scan_bounds(a, spans, dy)
    one = {k: w[..., 25:50] if k in ("u", "delta", "B", "C", "z") else w for k, w in a.items()}
    one["x0"] = a["x0"][2:]
    want = T.scan_bounds(one, S.dense_spans(1, 25), dy[..., 25:50])
    for k in ("y", "du", "ddelta", "dz", "dB", "dC"):
        assert np.array_equal(got[k][..., 25:50], want[k]) and (got[k][..., :5] == 0).all(), k
    for k in ("x", "dx0"):
        assert np.array_equal(got[k][2:], want[k]), k
