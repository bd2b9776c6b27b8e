"""Pins of the linear attention and layer norm oracle (CPU): against the selective
scan's oracle where both compute the same, the plain double sum, torch's layer norm,
and differences for every gradient; planted mistakes are caught."""
import numpy as np
import pytest

import oracle.linear_oracle as O
import oracle.selective_oracle as S


def _inputs(seed=0, Bsz=2, H=4, G=2, N=3, P=5, L=7):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return dict(q=n((Bsz, G, N, L)), k=n((Bsz, G, N, L)), v=n((Bsz, H, P, L)), g=-r.random((Bsz, H, L)),
                beta=r.random((Bsz, H, L)), D=n(H), scale=0.7, x0=n((Bsz, H, N, P)))


def _call(a, spans, **kw):
    a = {**a, **kw}
    return O.attention(a["q"], a["k"], a["v"], a["g"], a["beta"], a["D"], a["scale"], a["x0"], spans)


def test_is_the_selective_scan_with_one_decay_per_head():
    """A scan whose channels of a head share dt and one A for all states."""
    a = _inputs()
    Bsz, H, P, L = a["v"].shape
    N, G = a["q"].shape[2], a["q"].shape[1]
    rate = np.linspace(0.3, 2.0, H)
    dt = np.abs(a["beta"]) + 0.05
    flat = lambda v: v.reshape(Bsz, H * P, L)  # noqa: E731
    y, last, _ = S.scan(flat(a["v"]), flat(np.repeat(dt[:, :, None], P, 2)), np.repeat(-rate, P)[:, None] * np.ones(N), a["k"],
                        a["q"], np.repeat(a["D"], P), None, None, False,
                        a["x0"].transpose(0, 1, 3, 2).reshape(Bsz, H * P, N), S.dense_spans(Bsz, L))
    mine, x, _ = _call(a, S.dense_spans(Bsz, L), g=-dt * rate[:, None], beta=dt, scale=1.0)
    np.testing.assert_allclose(mine, y.reshape(Bsz, H, P, L), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(x, last.reshape(Bsz, H, P, N).transpose(0, 1, 3, 2), rtol=1e-12, atol=1e-12)


def test_is_the_double_sum():
    a = _inputs(1, Bsz=1)
    L = a["q"].shape[3]
    y, x, _ = _call(a, [(0, 0, L)])
    for h in range(4):
        c = np.cumsum(a["g"][0, h])
        w = np.tril(np.exp(c[:, None] - c)) * a["beta"][0, h]
        q, k, v = a["q"][0, h // 2].T, a["k"][0, h // 2].T, a["v"][0, h].T
        want = a["scale"] * ((q @ k.T * w) @ v + np.exp(c)[:, None] * (q @ a["x0"][0, h])) + a["D"][h] * v
        np.testing.assert_allclose(y[0, h].T, want, rtol=1e-12, atol=1e-12)
        end = np.exp(c[-1]) * a["x0"][0, h] + (k * w[-1][:, None]).T @ v
        np.testing.assert_allclose(x[0, h], end, rtol=1e-12, atol=1e-12)


def test_sequences_are_apart():
    a = _inputs(2, Bsz=1)
    a["x0"] = np.random.default_rng(3).standard_normal((3, 4, 3, 5))
    y, x, _ = _call(a, [(0, 0, 3), (0, 3, 3), (0, 4, 7)])
    assert np.isnan(y[..., 3]).all() and np.array_equal(x[1], a["x0"][1])
    part = {k: v[..., 4:7] if k in ("q", "k", "v", "g", "beta") else v for k, v in a.items()}
    alone, end, _ = _call(part, [(0, 0, 3)], x0=a["x0"][2:])
    np.testing.assert_array_equal(y[..., 4:7], alone)
    np.testing.assert_array_equal(x[2], end[0])


def _objective(a, dy, dx, spans, sign=1.0):
    y, x, _ = _call(a, spans)
    return np.nansum(y * dy) + (x * dx).sum()


@pytest.mark.parametrize("spans", [[(0, 0, 7), (1, 0, 7)], [(0, 0, 4), (1, 0, 0)]])
def test_gradients_against_differences(spans):
    a = _inputs(4)
    r = np.random.default_rng(5)
    dy, dx = r.standard_normal(a["v"].shape), r.standard_normal(a["x0"].shape)
    g = O.attention_grad(a["q"], a["k"], a["v"], a["g"], a["beta"], a["D"], a["scale"], a["x0"], dy, dx, spans)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("D", "dD"), ("x0", "dx0")):
        way, e = r.standard_normal(a[n].shape), 1e-6
        slope = (_objective({**a, n: a[n] + e * way}, dy, dx, spans) - _objective({**a, n: a[n] - e * way}, dy, dx, spans)) / (2 * e)
        assert abs(slope - np.nansum(g[d] * way)) <= 1e-7 * max(1.0, abs(slope)), d


def test_magnitudes_bound_the_sums():
    a = _inputs(6)
    spans = [(0, 0, 7), (1, 0, 7)]
    y, x, _ = _call(a, spans)
    my, mx, _ = O.attention(a["q"], a["k"], a["v"], a["g"], a["beta"], a["D"], a["scale"], a["x0"], spans, True)
    assert (np.abs(y) <= my + 1e-12).all() and (np.abs(x) <= mx + 1e-12).all()
    dy, dx = np.random.default_rng(7).standard_normal(a["v"].shape), np.ones_like(a["x0"])
    args = (a["q"], a["k"], a["v"], a["g"], a["beta"], a["D"], a["scale"], a["x0"], dy, dx, spans)
    g, m = O.attention_grad(*args), O.attention_grad(*args, mag=True)
    assert all((np.abs(g[k]) <= m[k] + 1e-12).all() for k in g)


def test_planted_mistakes_are_caught():
    a = _inputs(8)
    spans = [(0, 0, 7), (1, 0, 7)]
    y, _, _ = _call(a, spans)
    for wrong in (dict(q=a["k"], k=a["q"]), dict(g=np.roll(a["g"], 1, 2)), dict(beta=np.ones_like(a["beta"])),
                  dict(D=np.zeros(4)), dict(x0=a["x0"][::-1]), dict(scale=-0.7)):
        assert np.abs(_call(a, spans, **wrong)[0] - y).max() > 1e-3


# -------------------------------------------------------------- layer norm ----

def _norm_inputs(seed=0, Bsz=2, H=12, L=3):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return dict(u=n((Bsz, H, L)) + 0.3, weight=n(H), bias=n(H), z=n((Bsz, H, L)))


def test_norm_is_torchs():
    torch = pytest.importorskip("torch")
    a = _norm_inputs()
    t = lambda v: torch.from_numpy(v)  # noqa: E731
    y, _, _ = O.norm(a["u"], a["weight"], a["bias"], None, "after", False, 1, 1e-5)
    want = torch.nn.functional.layer_norm(t(a["u"]).transpose(1, 2), (12,), t(a["weight"]), t(a["bias"]), 1e-5)
    np.testing.assert_allclose(y, want.transpose(1, 2).numpy(), rtol=1e-12, atol=1e-12)
    y, _, _ = O.norm(a["u"], a["weight"], a["bias"], None, "after", False, 3, 1e-5)
    want = torch.nn.functional.group_norm(t(a["u"].transpose(0, 2, 1).reshape(6, 12)), 3, t(a["weight"]), t(a["bias"]), 1e-5)
    np.testing.assert_allclose(y, want.numpy().reshape(2, 3, 12).transpose(0, 2, 1), rtol=1e-12, atol=1e-12)
    y, _, _ = O.norm(a["u"], a["weight"], None, a["z"], "before", True, 1, 1e-5)
    s = torch.nn.functional.silu(t(a["z"])) * t(a["u"])
    want = torch.nn.functional.rms_norm(s.transpose(1, 2), (12,), t(a["weight"]), 1e-5)
    np.testing.assert_allclose(y, want.transpose(1, 2).numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("gate", ["", "before", "after"])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_against_differences(gate, rms):
    a = _norm_inputs(1)
    r = np.random.default_rng(2)
    dy = r.standard_normal(a["u"].shape)
    more = (gate or "after", rms, 2, 1e-5)
    f = lambda b: (O.norm(b["u"], b["weight"], b["bias"], b["z"] if gate else None, *more)[0] * dy).sum()  # noqa: E731
    g = O.norm_grad(a["u"], dy, a["weight"], a["bias"], a["z"] if gate else None, *more)
    for n in ("u", "weight", "bias") + (("z",) if gate else ()):
        way, e = r.standard_normal(a[n].shape), 1e-6
        slope = (f({**a, n: a[n] + e * way}) - f({**a, n: a[n] - e * way})) / (2 * e)
        assert abs(slope - (g["d" + n] * way).sum()) <= 1e-7 * max(1.0, abs(slope)), n
