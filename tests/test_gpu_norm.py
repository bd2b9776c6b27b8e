"""Layer norm on the GPU against the float64 oracle: types, storage orders, groups,
gates, odd and large sizes, gradients, single tokens, infinities, streams and graphs.

Tolerances count roundings in half steps of float32: the mean and the mean square
come from sums of at most 64 terms a thread and 30 more additions on the way together
(100 each, relative to magnitudes), a normed number and its products take 20, the gate's
exponential |z| + 16; and half a step of the output's type."""
import numpy as np
import pytest

import oracle.linear_oracle as O
from tests.selective_cases import HALF_STEP, SMALLEST, on_device, rounded, torch_type

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"
U = 2.0 ** -24


def _ssm():
    from structured_state_space_amd import ssm
    return ssm


def _np(t):
    return t.detach().double().cpu().numpy()


def _f32(a):
    return None if a is None else torch.from_numpy(np.asarray(a)).float().to(DEV)


def inputs(seed, name, Bsz, H, L, gate, bias=True, weight=True, shift=0.5):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    return dict(u=rounded(n(Bsz, H, L) + shift, name), dy=rounded(n(Bsz, H, L), name),
                z=rounded(n(Bsz, H, L), name) if gate else None, weight=rounded(n(H), "f32") if weight else None,
                bias=rounded(n(H), "f32") if bias else None)


def bounds(a, gate, rms, groups, eps):
    """Magnitudes, times U, of what rounding does to each output."""
    Bsz, H, L = a["u"].shape
    D = H // groups
    sig = lambda v: 0.5 * (1.0 + np.tanh(0.5 * v))  # noqa: E731
    z = a["z"]
    _, n, r = O.norm(a["u"], a["weight"], a["bias"], z, gate, rms, groups, eps)
    group = lambda v: v.reshape(Bsz, groups, D, L)  # noqa: E731
    flat = lambda v: v.reshape(Bsz, H, L)  # noqa: E731
    w = np.ones(H) if a["weight"] is None else np.abs(a["weight"])
    b = np.zeros(H) if a["bias"] is None else np.abs(a["bias"])
    s = 1.0 if z is None else np.abs(z) * sig(z)
    soft = 0.0 if z is None else np.abs(z) + 16.0            # roundings of the gate
    x = np.abs(a["u"]) * s if gate == "before" and z is not None else np.abs(a["u"])
    gx = soft if gate == "before" else 0.0
    # of a normed number: its own input's, the mean's, and the root's relative to itself
    mean = 0.0 if rms else group(x).mean(2, keepdims=True)
    worst = 0.0 if z is None else np.max(gx * np.ones_like(x))
    dn = flat(r * (group(x * (gx + 4.0)) + mean * (100.0 + worst))) + np.abs(n) * (220.0 + 2.0 * worst)
    y = dn * w[:, None] + 4.0 * (np.abs(n) * w[:, None] + b[:, None])
    out = dict(y=y if gate == "before" or z is None else s * (y + (soft + 2.0) * (np.abs(n) * w[:, None] + b[:, None])))
    d = np.abs(a["dy"])
    pre = np.abs(n) * w[:, None] + b[:, None]
    slope = 1.1 * np.ones_like(d) if z is not None else None
    ed = 1.0
    if z is not None and gate == "after":
        out["dz"] = d * (slope * y + (1.1 * soft + 12.0) * pre)
        d, ed = d * s, soft + 2.0
    sums = 100.0 + Bsz * L / 2.0 ** 6                        # of a column's partial sums
    out["dweight"] = (d * (dn + (ed + sums) * np.abs(n))).sum((0, 2))
    out["dbias"] = (d * (ed + sums)).sum((0, 2))
    g, m, e = group(d * w[:, None]), group(np.abs(n)), group(dn)
    e_g = np.max(ed * np.ones_like(d)) + 2.0
    inner = (g * m).mean(2, keepdims=True)
    da = g * e_g + m * ((g * e).mean(2, keepdims=True) + (100.0 + e_g) * inner) + e * inner
    mag = g + m * inner
    if not rms:
        da, mag = da + (100.0 + e_g) * g.mean(2, keepdims=True), mag + g.mean(2, keepdims=True)
    da, mag = flat(r * (da + (230.0 + 2.0 * worst) * mag)), flat(r * mag)
    if z is not None and gate == "before":
        out["dz"] = np.abs(a["u"]) * (1.1 * da + (1.1 * soft + 12.0) * mag)
        da = s * (da + (soft + 2.0) * mag)
    out["du"] = da
    return {k: U * v for k, v in out.items()}


def check(a, name, order, groups=1, rms=False, gate="after", eps=1e-5):
    ssm = _ssm()
    u, z, dy = (None if a[k] is None else on_device(a[k], name, order) for k in ("u", "z", "dy"))
    more = dict(weight=_f32(a["weight"]), bias=_f32(a["bias"]), z=z, gate=gate, rms=rms, groups=groups, eps=eps)
    out = ssm.layer_norm(u, **more)
    out.update(ssm.layer_norm_backward(u, dy, **more))
    torch.cuda.synchronize()
    e = float(np.float32(eps))
    want = O.norm_grad(a["u"], a["dy"], a["weight"], a["bias"], a["z"], gate, rms, groups, e)
    want["y"] = O.norm(a["u"], a["weight"], a["bias"], a["z"], gate, rms, groups, e)[0]
    err = bounds(a, gate, rms, groups, e)
    for k, v in out.items():
        if v is None:
            assert k == "dz" and z is None or k == "dweight" and a["weight"] is None or k == "dbias" and a["bias"] is None
            continue
        kind = "f32" if k in ("dweight", "dbias") else name
        x, w, b = _np(v), want[k], err[k]
        tol = HALF_STEP[kind] * (np.abs(w) + b) + b + SMALLEST[kind]
        bad = ~(np.abs(x - w) <= tol)
        if bad.any():
            at = tuple(int(i[0]) for i in np.nonzero(bad))
            raise AssertionError(f"{k}: {int(bad.sum())} of {bad.size} off, first at {at}: {x[at]} for {w[at]}, tolerance {tol[at]:.3g}")


CASES = [  # channels, groups, rms, gate
    (1, 1, True, ""), (1, 1, False, "after"), (7, 7, True, "before"), (48, 3, False, "after"), (64, 1, True, "before"), (65, 1, False, ""),
    (120, 1, True, "after"), (256, 2, False, "before"), (257, 1, True, ""), (500, 1, False, "after"), (1000, 1, True, "before"),
    (1025, 1, False, ""), (2048, 1, True, "before"), (2500, 1, False, "after"), (4104, 1, True, ""),
]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["tokens", "rows", "sliced", "mixed"])
@pytest.mark.parametrize("H,groups,rms,gate", CASES)
def test_norm(name, order, H, groups, rms, gate):
    L = 67 if H < 300 else 5
    check(inputs(H, name, 2, H, L, gate, bias=H % 2 == 0, weight=H % 3 != 0), name, order, groups, rms, gate or "after")


@pytest.mark.parametrize("H", [9000, 17000, 33000])
@pytest.mark.parametrize("order", ["tokens", "rows"])
def test_many_channels(H, order):
    check(inputs(H, "bf16", 1, H, 3, "before"), "bf16", order, 1, False, "before")


@pytest.mark.parametrize("order", ["tokens", "rows"])
@pytest.mark.parametrize("H,groups", [(64, 1), (96, 12), (1536, 1), (4096, 1)])
def test_many_steps(order, H, groups):
    """Workgroups go over several steps, and their parts of the parameters' gradients are added up."""
    check(inputs(3, "f32", 3, H, 700 if H < 200 else 500, "", shift=0.0), "f32", order, groups, False)


@pytest.mark.parametrize("name,H,groups,L", [("f32", 24, 1, 17000), ("bf16", 100, 1, 9000), ("f16", 200, 1, 4500),
                                              ("f32", 384, 1, 2200), ("bf16", 700, 1, 2200), ("f32", 96, 4, 5000),
                                              ("bf16", 9000, 1, 520), ("f32", 9000, 1, 260)])
def test_more_steps_than_workgroups_have_at_once(name, H, groups, L):
    """... also where a workgroup has several steps at a time and joins their sums at the end."""
    check(inputs(5, name, 1, H, L, "before", shift=0.0), name, "tokens", groups, True, "before")


def test_far_from_zero():
    """The mean is taken before the squares: 2^12 standard deviations away the variance is still there (each input is
    rounded to 2^-24 of the shift, and the bounds say what that leaves)."""
    a = inputs(4, "f32", 2, 600, 9, "", shift=0.0)
    a["u"] = rounded(a["u"] + 4096.0, "f32")
    for order in ("tokens", "rows"):
        check(a, "f32", order)


def test_constant_rows_and_eps():
    """A row without variance gives the bias; eps of zero is allowed where there is one."""
    ssm = _ssm()
    u = torch.full((1, 40, 6), 3.25, device=DEV)
    bias = torch.randn(40, device=DEV)
    y = ssm.layer_norm(u, bias=bias)["y"]
    assert torch.equal(y, bias[None, :, None].expand(1, 40, 6))
    check(inputs(5, "f32", 1, 40, 6, ""), "f32", "tokens", eps=0.0)


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_tokens_of_a_decode_batch(name):
    """[Bsz, H]: the same as one step of [Bsz, H, 1], in rows any number of elements apart."""
    ssm = _ssm()
    a = inputs(6, name, 5, 96, 1, "after")
    w, b = _f32(a["weight"]), _f32(a["bias"])
    for order in ("rows", "sliced"):
        u, z, dy = (on_device(a[k], name, order) for k in ("u", "z", "dy"))
        want = ssm.layer_norm(u, w, b, z=z, groups=4)["y"][..., 0]
        got = ssm.layer_norm(u[..., 0], w, b, z=z[..., 0], groups=4)["y"]
        assert got.shape == (5, 96) and torch.equal(got, want)
        g = ssm.layer_norm_backward(u[..., 0], dy[..., 0], w, b, z=z[..., 0], groups=4)
        h = ssm.layer_norm_backward(u, dy, w, b, z=z, groups=4)
        assert torch.equal(g["du"], h["du"][..., 0]) and torch.equal(g["dz"], h["dz"][..., 0]) and torch.equal(g["dweight"], h["dweight"])
    y = torch.empty((5, 96), dtype=torch_type(name), device=DEV)
    assert ssm.layer_norm(u[..., 0], w, b, z=z[..., 0], groups=4, y=y)["y"] is y and torch.equal(y, want)


@pytest.mark.parametrize("order", ["tokens", "rows"])
def test_infinite_inputs_stay_in_their_step_and_group(order):
    ssm = _ssm()
    a = inputs(7, "bf16", 2, 64, 70, "before")
    u, z, dy = (on_device(a[k], "bf16", order) for k in ("u", "z", "dy"))
    w = _f32(a["weight"])
    call = lambda: (ssm.layer_norm(u, w, z=z, gate="before", groups=4)["y"].clone(),  # noqa: E731
                    ssm.layer_norm_backward(u, dy, w, z=z, gate="before", groups=4)["du"].clone())
    want = call()
    for bad in (float("inf"), float("nan")):
        u[1, 20, 33] = bad
        got = call()
        keep = torch.ones((2, 64, 70), dtype=torch.bool, device=DEV)
        keep[1, 16:32, 33] = False
        for p, q in zip(got, want):
            assert torch.equal(p[keep], q[keep]) and not torch.isfinite(p[1, 20, 33].float())


def test_broadcast_gate_and_large_strides():
    ssm = _ssm()
    a = inputs(8, "bf16", 2, 64, 5, "after")
    u, dy, w = on_device(a["u"], "bf16", "tokens"), on_device(a["dy"], "bf16", "tokens"), _f32(a["weight"])
    z = on_device(a["z"], "bf16", "tokens")[..., :1].expand(2, 64, 5)
    whole = z.transpose(1, 2).contiguous().transpose(1, 2)
    for p, q in ((z, whole),):
        assert torch.equal(ssm.layer_norm(u, w, z=p)["y"], ssm.layer_norm(u, w, z=q)["y"])
        g, h = (ssm.layer_norm_backward(u, dy, w, z=v) for v in (p, q))
        assert all(torch.equal(g[k], h[k]) for k in ("du", "dz", "dweight"))
    big = torch.empty((1 << 31) + (1 << 26), dtype=torch.bfloat16, device=DEV)
    far = torch.as_strided(big, u.shape, ((1 << 31) - 9, 1, (1 << 23) - 1)).copy_(u)
    assert torch.equal(ssm.layer_norm(far, w)["y"], ssm.layer_norm(u, w)["y"])
    assert torch.equal(ssm.layer_norm_backward(far, dy, w)["du"], ssm.layer_norm_backward(u, dy, w)["du"])


def test_repeats_streams_and_workspaces():
    ssm = _ssm()
    a = inputs(9, "bf16", 3, 320, 200, "before")
    u, z, dy = (on_device(a[k], "bf16", "tokens") for k in ("u", "z", "dy"))
    w, b = _f32(a["weight"]), _f32(a["bias"])
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV)

    def step(workspace=None):
        g = ssm.layer_norm_backward(u, dy, w, b, z=z, gate="before", workspace=workspace)
        return [ssm.layer_norm(u, w, b, z=z, gate="before")["y"], *g.values()]

    want = step()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    got += [step(ws), step(ws)]
    assert all(torch.equal(p, q) for g in got for p, q in zip(g, want))
    for bad in (torch.empty(8, dtype=torch.uint8, device=DEV), ws.cpu()):
        with pytest.raises(ValueError):
            step(bad)


def test_without_parameters_nothing_is_summed():
    ssm = _ssm()
    a = inputs(10, "f32", 1, 64, 40, "", bias=False, weight=False)
    u, dy = on_device(a["u"], "f32", "tokens"), on_device(a["dy"], "f32", "tokens")
    g = ssm.layer_norm_backward(u, dy)
    assert g["dweight"] is None and g["dbias"] is None and g["dz"] is None


def test_refusals_name_the_argument():
    ssm = _ssm()
    u = torch.randn((2, 64, 5), device=DEV)
    w = torch.ones(64, device=DEV)
    for kw, name in [(dict(weight=w[:3]), "weight"), (dict(bias=w.half()), "bias"), (dict(z=u[:1]), "z"), (dict(z=u.half()), "z"),
                     (dict(gate="both"), "gate"), (dict(y=u[:, :4]), "y")]:
        with pytest.raises(ValueError, match=f"^{name}"):
            ssm.layer_norm(u, **kw)
    with pytest.raises(ValueError, match="^dy"):
        ssm.layer_norm_backward(u, u[:1])
    for kw in (dict(groups=5), dict(groups=0), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(ssm.SSMError):
            ssm.layer_norm(u, **kw)
    with pytest.raises(ssm.SSMError):      # an output that shares places
        ssm.layer_norm(u, y=torch.empty((2, 64, 1), device=DEV).expand(2, 64, 5))
