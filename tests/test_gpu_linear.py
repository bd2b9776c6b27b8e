"""Linear attention on the GPU against the float64 oracle: types, storage orders,
head groups, odd sizes, ragged and packed sequences, states and slots, gradients,
single tokens, resets, infinities, streams and captured graphs.

Tolerances count roundings (tests/linear_cases.py)."""
import numpy as np
import pytest

import oracle.linear_oracle as O
import oracle.selective_oracle as S
from tests import linear_cases as K

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"
FORWARD, BACKWARD = ("y", "x"), ("dq", "dk", "dv", "dg", "dbeta", "dD", "dx0")


def _ssm():
    from structured_state_space_amd import ssm
    return ssm


def _np(t):
    return t.detach().double().cpu().numpy()


def _f32(a):
    return None if a is None else torch.from_numpy(np.asarray(a)).float().to(DEV)


def _int(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def _given(offsets=None, lengths=None):
    return dict(offsets=None if offsets is None else _int(offsets), lengths=None if lengths is None else _int(lengths))


def check(a, name, order, offsets=None, lengths=None, grads=True, save=True):
    """Forward and backward of a call against the oracle; what was not written keeps its value."""
    ssm = _ssm()
    Bsz, _, _, L = a["v"].shape
    spans = S.dense_spans(Bsz, L, lengths) if offsets is None else S.packed_spans(offsets)
    args, kw = K.call_args(a, name, order)
    kw.update(_given(offsets, lengths))
    y = torch.full_like(args[2], 7.0)
    f = ssm.linear_attention(*args, **kw, want_state=True, save=grads and save, y=y)
    assert f["y"] is y
    torch.cuda.synchronize()
    want, mag = K.forward(a, spans), K.forward(a, spans, True)
    K.assert_all({k: _np(f[k]) for k in FORWARD}, want, mag, a, name, spans, "forward")
    assert (_np(y)[np.isnan(want["y"])] == 7.0).all()
    if not grads:
        return
    dy = K.on_device(a["dy"], name, order)
    g = ssm.linear_attention_backward(*args, dy, dx=_f32(a["dx"]), saved=f["saved"], **kw)
    torch.cuda.synchronize()
    want, mag = K.backward(a, spans), K.backward(a, spans, True)
    got = {k: _np(v) for k, v in g.items() if v is not None}
    assert set(got) == {k for k in BACKWARD if not (k == "dbeta" and a["beta"] is None or k == "dD" and a["D"] is None
                                                    or k == "dx0" and a["x0"] is None)}
    K.assert_all(got, want, mag, a, name, spans, "backward")
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        if n in got:
            assert (got[n][np.isnan(want[n])] == 0.0).all(), n


SIZES = [  # Bsz, H, G, N, P, L
    (1, 1, 1, 1, 1, 1), (1, 1, 1, 16, 16, 2), (2, 3, 1, 17, 5, 31), (1, 2, 2, 32, 64, 32), (1, 2, 1, 33, 65, 33),
    (2, 4, 2, 64, 64, 64), (1, 4, 1, 64, 64, 65), (1, 2, 1, 128, 64, 127), (1, 2, 2, 128, 128, 129), (1, 1, 1, 129, 63, 200),
    (1, 2, 1, 256, 80, 150), (3, 2, 1, 200, 256, 70), (1, 6, 3, 40, 24, 300),
]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(name, size):
    check(K.inputs(1, name, *size), name, "tokens")


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["rows", "sliced", "mixed"])
@pytest.mark.parametrize("size", [(2, 2, 1, 64, 64, 128), (1, 2, 2, 40, 72, 90), (1, 1, 1, 130, 33, 67)])
def test_orders(name, order, size):
    check(K.inputs(2, name, *size), name, order)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["tokens", "rows"])
@pytest.mark.parametrize("size", [(1, 44, 1, 24, 16, 70), (1, 80, 2, 64, 64, 40), (1, 41, 1, 128, 70, 66), (1, 36, 1, 250, 130, 65)])
def test_many_heads_of_a_group(name, order, size):
    """A workgroup has several heads one after the other for the gradients of q and k, with one to three blocks of
    values each, and not as many in the last."""
    check(K.inputs(22, name, *size), name, order)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("beta,skip,carry", [(False, False, False), (True, False, True), (False, True, False)])
def test_without_what_is_optional(name, beta, skip, carry):
    check(K.inputs(3, name, 2, 4, 2, 48, 40, 100, beta=beta, skip=skip, carry=carry), name, "tokens")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["tokens", "rows"])
def test_packed_and_ragged(name, order):
    offsets = [0, 1, 1, 66, 194, 260]
    check(K.inputs(4, name, 1, 2, 1, 64, 48, 270, S=5), name, order, offsets=offsets)
    check(K.inputs(5, name, 4, 2, 1, 32, 64, 130), name, order, lengths=[130, 0, 64, 1])


def test_many_packed_sequences():
    """More sequences than a wave searches at once, many of them empty."""
    r = np.random.default_rng(6)
    lens = r.integers(0, 4, 150) * r.integers(0, 2, 150)
    offsets = np.concatenate([[2], 2 + np.cumsum(lens)])
    a = K.inputs(6, "bf16", 1, 2, 1, 32, 32, int(offsets[-1]) + 3, S=150)
    check(a, "bf16", "tokens", offsets=offsets.tolist())


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lengths", [None, [700, 300]])
def test_segments(name, lengths):
    """Few heads on a long row: the walk is cut, the state goes from piece to piece."""
    ssm = _ssm()
    a = K.inputs(7, name, 2, 1, 1, 32, 32, 700, pace=0.03)
    assert ssm.linear_bytes(ssm.OP_LINEAR_ATTENTION, K.torch_type(name), 2, 1, 32, 32, 1, 700) > 0
    check(a, name, "tokens", lengths=lengths)
    check(K.inputs(8, name, 1, 1, 1, 32, 32, 700, S=3, pace=0.03), name, "tokens", offsets=[5, 400, 400, 690])


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_descending_offsets_stay_within_the_workspace(name):
    """They make more pieces than the workspace has places: what they name is unspecified, the rest is not.
    Two sequences of 700 steps and an empty one are cut into seven pieces (float32: thirteen), places
    are for those of 700 steps and one more for each sequence."""
    ssm = _ssm()
    a = K.inputs(21, name, 1, 1, 1, 32, 32, 700, S=3, pace=0.03)
    args, kw = K.call_args(a, name, "tokens")
    tidy = torch.tensor([0, 700, 700, 700], dtype=torch.int32, device=DEV)
    wrong = torch.tensor([0, 700, 0, 700], dtype=torch.int32, device=DEV)
    want = ssm.linear_attention(*args, **kw, offsets=tidy, want_state=True)["x"]
    need = ssm.linear_bytes(ssm.OP_LINEAR_ATTENTION, K.torch_type(name), 1, 1, 32, 32, 1, 700, S=3, packed=True)
    assert need > 0
    ws = torch.full((need + (1 << 16),), 77, dtype=torch.uint8, device=DEV)
    out = ssm.linear_attention(*args, **kw, offsets=wrong, want_state=True, save=True, workspace=ws)
    assert bool((ws[need:] == 77).all())
    assert torch.equal(out["x"][0], want[0])
    dy = K.on_device(a["dy"], name, "tokens")
    need = ssm.linear_bytes(ssm.OP_LINEAR_ATTENTION_BACKWARD, K.torch_type(name), 1, 1, 32, 32, 1, 700, S=3, packed=True)
    ws = torch.full((need + (1 << 16),), 77, dtype=torch.uint8, device=DEV)
    ssm.linear_attention_backward(*args, dy, dx=_f32(a["dx"]), saved=out["saved"], offsets=wrong, workspace=ws, **kw)
    assert bool((ws[need:] == 77).all())


def test_backward_computes_the_states_again():
    ssm = _ssm()
    a = K.inputs(9, "bf16", 2, 4, 2, 64, 64, 200)
    args, kw = K.call_args(a, "bf16", "tokens")
    dy = K.on_device(a["dy"], "bf16", "tokens")
    f = ssm.linear_attention(*args, **kw, save=True)
    one = ssm.linear_attention_backward(*args, dy, dx=_f32(a["dx"]), saved=f["saved"], **kw)
    two = ssm.linear_attention_backward(*args, dy, dx=_f32(a["dx"]), **kw)
    assert all(torch.equal(one[k], two[k]) for k in BACKWARD)


def test_repeated_calls_give_the_same_bits_and_workspaces_are_free_to_choose():
    ssm = _ssm()
    a = K.inputs(10, "bf16", 1, 8, 1, 64, 64, 500)
    args, kw = K.call_args(a, "bf16", "tokens")
    dy = K.on_device(a["dy"], "bf16", "tokens")
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)   # NaN in every float

    def both(workspace=None):
        f = ssm.linear_attention(*args, **kw, want_state=True, save=True, workspace=workspace)
        g = ssm.linear_attention_backward(*args, dy, dx=_f32(a["dx"]), saved=f["saved"], workspace=workspace, **kw)
        return [f["y"], f["x"], *(g[k] for k in BACKWARD)]

    want = both()
    for w in (None, ws, ws):
        assert all(torch.equal(p, q) for p, q in zip(both(w), want))
    small = torch.empty(64, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        ssm.linear_attention(*args, **kw, workspace=small)
    with pytest.raises(ValueError):
        ssm.linear_attention_backward(*args, dy, workspace=small, **kw)
    with pytest.raises(ValueError):
        ssm.linear_attention(*args, **kw, workspace=ws.cpu())


def test_final_states_may_replace_the_initial_ones():
    """In place and in a pool of slots, whole and in segments; a slot outside the pool is skipped."""
    ssm = _ssm()
    for H, L, pace in ((3, 90, 0.2), (1, 900, 0.02)):
        a = K.inputs(11, "bf16", 3, H, 1, 32, 48, L, pace=pace)
        args, kw = K.call_args(a, "bf16", "tokens")
        want = ssm.linear_attention(*args, **kw, want_state=True)
        x = _f32(a["x0"])
        got = ssm.linear_attention(*args, **{**kw, "x0": x}, x_out=x)
        assert got["x"] is x and torch.equal(x, want["x"]) and torch.equal(got["y"], want["y"])
        pool = torch.full((5, H, 32, 48), 3.0, device=DEV)
        pool[4], pool[1] = _f32(a["x0"])[0], _f32(a["x0"])[2]
        y = torch.full_like(args[2], 7.0)
        got = ssm.linear_attention(*args, **{**kw, "x0": pool}, x_out=pool, slots=_int([4, -1, 1]), y=y)
        assert torch.equal(pool[4], want["x"][0]) and torch.equal(pool[1], want["x"][2])
        assert bool((pool[[0, 2, 3]] == 3.0).all())
        assert torch.equal(y[[0, 2]], want["y"][[0, 2]]) and bool((y[1] == 7.0).all())


def test_slots_without_states():
    ssm = _ssm()
    a = K.inputs(12, "bf16", 3, 2, 1, 32, 32, 40, carry=False)
    args, kw = K.call_args(a, "bf16", "tokens")
    y = torch.full_like(args[2], 7.0)
    ssm.linear_attention(*args, **kw, slots=_int([2 ** 20, -1, 0]), y=y)
    want = ssm.linear_attention(*args, **kw)["y"]
    assert torch.equal(y[[0, 2]], want[[0, 2]]) and bool((y[1] == 7.0).all())


# ----------------------------------------------- decays and extreme values ----

@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_fixed_decays_are_broadcast(name):
    ssm = _ssm()
    a = K.inputs(13, name, 2, 4, 2, 32, 32, 150, beta=False)
    a["g"] = np.broadcast_to(np.array([-0.01, -0.3, 0.0, -2.0])[None, :, None], (2, 4, 150))
    a["g"] = K.rounded(a["g"], "f32")
    args, kw = K.call_args(a, name, "tokens")
    fixed = _f32(a["g"][0, :, 0])[None, :, None].expand(2, 4, 150)
    assert fixed.stride() == (0, 1, 0)
    dy = K.on_device(a["dy"], name, "tokens")
    f, w = (ssm.linear_attention(*args[:3], g, **kw, want_state=True, save=True) for g in (fixed, args[3]))
    assert torch.equal(f["y"], w["y"]) and torch.equal(f["x"], w["x"])
    got = ssm.linear_attention_backward(*args[:3], fixed, dy, saved=f["saved"], **kw)
    spans = S.dense_spans(2, 150)
    K.assert_all({k: _np(got[k]) for k in BACKWARD if got[k] is not None}, K.backward({**a, "dx": None}, spans),
                 K.backward({**a, "dx": None}, spans, True), a, name, spans)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_resets(name):
    """g of minus infinity: nothing from before is left, at a chunk's start, within one, twice in a row, at the first
    and the last step; its own gradient is zero."""
    a = K.inputs(14, name, 1, 2, 1, 32, 48, 200)
    for t in (0, 10, 11, 64, 100, 128, 199):
        a["g"][0, 0, t] = -np.inf
    a["g"][0, 1, 70:90] = -50.0     # decays that underflow together
    check(a, name, "tokens")
    args, kw = K.call_args(a, name, "tokens")
    dg = _ssm().linear_attention_backward(*args, K.on_device(a["dy"], name, "tokens"), **kw)["dg"]
    assert bool((dg[0, 0, [0, 10, 11, 64, 100, 128, 199]] == 0.0).all())


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_growth(name):
    """Positive g: within the documented sums by products, beyond them step by step (forward)."""
    a = K.inputs(15, name, 1, 2, 1, 32, 32, 140, carry=False, beta=False)
    a["g"] = K.rounded(np.where(np.arange(140) % 3 == 0, 0.05, -0.04)[None, None] * np.array([1.0, -0.5])[None, :, None], "f32")
    check(a, name, "tokens")
    a["g"][0, 0, 64:96] = 1.5       # 48 over half a chunk
    a["g"][0, 0, 96:] = -1.5
    check(a, name, "tokens", grads=False)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_infinite_inputs_reach_nothing_before_them(name, bad, where):
    """... and of v their own value alone, of q their own step."""
    ssm = _ssm()
    a = K.inputs(16, name, 1, 4, 2, 32, 40, 150)
    args, kw = K.call_args(a, name, "tokens")
    clean = ssm.linear_attention(*args, **kw)["y"].clone()
    t, h = 90, 1
    args[dict(q=0, k=1, v=2)[where]][0, h // 2 if where != "v" else h, 7, t] = bad
    out = ssm.linear_attention(*args, **kw, want_state=True)
    y, x = out["y"], out["x"]
    others = [2, 3] if where != "v" else [0, 2, 3]
    near = lambda p, q: torch.allclose(p.float(), q.float(), rtol=2.0 ** -5, atol=2.0 ** -4)  # noqa: E731
    assert torch.equal(y[:, others], clean[:, others])
    # (the chunk goes step by step: other roundings than the products, of 2^-8 against magnitudes of up to 8)
    assert near(y[0, :, :, :t], clean[0, :, :, :t])
    if where == "q":
        assert near(y[0, :, :, t + 1:], clean[0, :, :, t + 1:]) and bool(torch.isfinite(x).all())
        assert not torch.isfinite(y[0, :2, :, t].float()).any()
    elif where == "v":
        rest = [i for i in range(40) if i != 7]
        assert near(y[0, h, rest], clean[0, h, rest]) and bool(torch.isfinite(x[0, h][:, rest]).all())
        assert not torch.isfinite(y[0, h, 7, t:].float()).any()
    else:
        assert not torch.isfinite(y[0, :2, :, t:].float()).any()
        rows = [i for i in range(32) if i != 7]
        assert bool(torch.isfinite(x[0, :2][:, rows]).all()) and not torch.isfinite(x[0, :2, 7]).any()


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_infinite_inputs_in_one_sequence_leave_the_others(name):
    ssm = _ssm()
    a = K.inputs(17, name, 1, 2, 1, 32, 32, 200, S=3)
    args, kw = K.call_args(a, name, "tokens")
    kw["offsets"] = _int([0, 70, 130, 200])
    dy = K.on_device(a["dy"], name, "tokens")

    def both():
        f = ssm.linear_attention(*args, **kw, want_state=True, save=True)
        g = ssm.linear_attention_backward(*args, dy, dx=_f32(a["dx"]), saved=f["saved"], **kw)
        return f, g

    f0, g0 = both()
    args[2][0, 0, 3, 100] = float("nan")
    args[3][0, 1, 110] = float("nan")
    f1, g1 = both()
    for t in (slice(0, 70), slice(130, 200)):
        assert torch.equal(f0["y"][..., t], f1["y"][..., t])
        assert all(torch.equal(g0[k][..., t], g1[k][..., t]) for k in ("dq", "dk", "dv", "dg", "dbeta"))
    assert torch.equal(f0["x"][[0, 2]], f1["x"][[0, 2]]) and torch.equal(g0["dx0"][[0, 2]], g1["dx0"][[0, 2]])


@pytest.mark.parametrize("size", [1e-6, 1e-3, 100.0])
def test_float16_of_any_size(size):
    """Products far outside float16's range of numbers, in results that are within it."""
    a = K.inputs(18, "f16", 1, 2, 1, 64, 64, 150, scale=1.0)
    q, k = (1.0, size) if size < 1 else (size, 1.0)
    a["q"], a["k"] = K.rounded(a["q"] * q, "f16"), K.rounded(a["k"] * k, "f16")
    for n in ("x0", "dx"):
        a[n] = K.rounded(a[n] * k, "f32")
    if size > 1:
        a["v"], a["dy"], a["D"] = K.rounded(a["v"] * 1e-2, "f16"), K.rounded(a["dy"] * 1e-2, "f16"), None
        a["x0"] = K.rounded(a["x0"] * 1e-2, "f32")
    check(a, "f16", "tokens")


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_nothing_outside_the_sequences_is_read(name):
    ssm = _ssm()
    a = K.inputs(19, name, 1, 2, 1, 64, 64, 150, S=2)
    a["dx"] = None
    args, kw = K.call_args(a, name, "tokens")
    kw["offsets"] = _int([10, 60, 140])
    dy = K.on_device(a["dy"], name, "tokens")

    def both():
        f = ssm.linear_attention(*args, **kw, want_state=True, save=True)
        g = ssm.linear_attention_backward(*args, dy, saved=f["saved"], **kw)
        return [f["y"][..., 10:140], f["x"], *(g[k] for k in BACKWARD)]

    want = [v.clone() for v in both()]
    for t in [*args, dy, kw["beta"]]:
        t[..., :10] = float("nan")
        t[..., 140:] = float("inf")
    assert all(torch.equal(p, q) for p, q in zip(both(), want))


def test_gradients_match_differences_of_the_kernel():
    ssm = _ssm()
    a = K.inputs(20, "f32", 1, 2, 1, 16, 16, 70)
    args, kw = K.call_args(a, "f32", "tokens")
    dy, dx = K.on_device(a["dy"], "f32", "tokens"), _f32(a["dx"])
    g = ssm.linear_attention_backward(*args, dy, dx=dx, **kw)
    named = dict(dq=args[0], dk=args[1], dv=args[2], dg=args[3], dbeta=kw["beta"], dD=kw["D"], dx0=kw["x0"])

    def objective():
        f = ssm.linear_attention(*args, **kw, want_state=True)
        return float((f["y"].double() * dy.double()).sum() + (f["x"].double() * dx.double()).sum())

    gen = torch.Generator(device=DEV).manual_seed(21)
    for n, t in named.items():
        way, e, keep = torch.randn(t.shape, generator=gen, device=DEV), 2.0 ** -9, t.clone()
        t.copy_(keep + e * way)
        up, wu = objective(), t.double() - keep.double()
        t.copy_(keep - e * way)
        down, wd = objective(), t.double() - keep.double()
        t.copy_(keep)
        # e^2 of the third difference; 2^-24 of the objective's magnitude (about 70 x 32 terms) over 2 e
        slope = float((g[n].double() * (wu - wd)).sum()) / (2 * e)
        assert abs((up - down) / (2 * e) - slope) <= 2e-2 * max(1.0, abs(slope)) ** 1.0 + 5e-2, n


# ------------------------------------------------------------ single tokens ----

@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1), (3, 4, 2, 16, 16), (2, 300, 1, 64, 64), (1, 3, 1, 33, 35), (2, 2, 2, 256, 256),
                                  (1, 8, 1, 128, 20), (5, 130, 1, 48, 80)])
def test_step(name, size):
    ssm = _ssm()
    Bsz, H, G, N, P = size
    a = K.inputs(22, name, Bsz, H, G, N, P, 1)
    spans = S.dense_spans(Bsz, 1)
    args, kw = K.call_args(a, name, "rows")
    x = kw.pop("x0")
    kw["beta"] = kw["beta"][..., 0]
    out = ssm.linear_attention_step(*(t[..., 0] for t in args), x, **kw)
    assert out["x"] is x
    K.assert_all(dict(y=_np(out["y"])[..., None], x=_np(x)), K.forward(a, spans), K.forward(a, spans, True), a, name, spans)


def test_step_slots_strides_and_resets():
    ssm = _ssm()
    Bsz, H, G, N, P = 4, 6, 3, 24, 20
    a = K.inputs(23, "bf16", Bsz, H, G, N, P, 1)
    a["g"][2, 4, 0] = -np.inf
    args, kw = K.call_args(a, "bf16", "mixed")
    pool = torch.full((9, H, N, P), 5.0, device=DEV)
    slots = [3, 9, 0, 8]
    for b, s in enumerate(slots):
        if s < 9:
            pool[s] = kw["x0"][b]
    y = torch.full((Bsz, P, H), 7.0, device=DEV, dtype=torch.bfloat16).transpose(1, 2)
    g, beta = args[3][..., 0].t().contiguous().t(), kw["beta"][..., 0]
    ssm.linear_attention_step(*(t[..., 0] for t in args[:3]), g, pool, beta=beta, D=kw["D"], scale=kw["scale"], slots=_int(slots),
                              y=y)
    spans = S.dense_spans(Bsz, 1)
    want, mag = K.forward(a, spans), K.forward(a, spans, True)
    run = [0, 2, 3]
    K.assert_all(dict(y=_np(y)[run][..., None], x=_np(pool[[3, 0, 8]])), {k: v[run] for k, v in want.items()},
                 {k: v[run] for k, v in mag.items()}, a, "bf16", spans)
    assert bool((y[1] == 7.0).all()) and bool((pool[[1, 2, 4, 5, 6, 7]] == 5.0).all())


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_prompt_then_tokens(name):
    """A prompt's states move on token by token as if the prompt had been longer."""
    ssm = _ssm()
    a = K.inputs(24, name, 2, 4, 2, 64, 64, 80)
    spans = S.dense_spans(2, 80)
    args, kw = K.call_args(a, name, "tokens")
    beta = kw.pop("beta")
    head = [t[..., :70] for t in args]
    f = ssm.linear_attention(*head, beta=beta[..., :70], **kw, want_state=True)
    x, ys = f["x"], [f["y"]]
    kw.pop("x0")
    for t in range(70, 80):
        ys.append(ssm.linear_attention_step(*(v[..., t] for v in args), x, beta=beta[..., t], **kw)["y"][..., None])
    K.assert_all(dict(y=_np(torch.cat(ys, -1)), x=_np(x)), K.forward(a, spans), K.forward(a, spans, True), a, name, spans)


# ----------------------------------------------- large strides and streams ----

def test_offsets_past_32_bits():
    """Rows, heads and steps whose places pass 2^31 elements."""
    ssm = _ssm()
    a = K.inputs(25, "bf16", 2, 2, 1, 32, 32, 70)
    args, kw = K.call_args(a, "bf16", "tokens")
    want = ssm.linear_attention(*args, **kw, want_state=True, save=True)
    dy = K.on_device(a["dy"], "bf16", "tokens")
    back = ssm.linear_attention_backward(*args, dy, saved=want["saved"], **kw)
    big = torch.empty((1 << 31) + (1 << 27), dtype=torch.bfloat16, device=DEV)
    far = lambda t, row, step: torch.as_strided(  # noqa: E731
        big, t.shape, (row, 1 << 12, 1, step) if t.shape[1] > 1 else (row, 0, 1, step)).copy_(t)
    for row, step in (((1 << 31) - 5, 1 << 14), (1 << 13, (1 << 23) - 8)):
        if row > 1 << 30:
            for i in range(3):
                moved = list(args)
                moved[i] = far(args[i], row, step)
                got = ssm.linear_attention(*moved, **kw, want_state=True)
                assert torch.equal(got["y"], want["y"]) and torch.equal(got["x"], want["x"])
            got = ssm.linear_attention_backward(*args, far(dy, row, step), saved=want["saved"], **kw)
        else:
            got = ssm.linear_attention_backward(args[0], args[1], far(args[2], row, step), *args[3:], dy, saved=want["saved"], **kw)
        assert all(torch.equal(got[k], back[k]) for k in BACKWARD if got[k] is not None)


def test_pool_past_32_bits():
    ssm = _ssm()
    H, N, P = 4, 128, 128
    rows = (1 << 32) // (H * N * P) // 4 + 40      # states past 2^31 bytes and 2^30 floats
    pool = torch.empty((rows, H, N, P), device=DEV)
    a = K.inputs(26, "bf16", 1, H, 1, N, P, 1)
    args, kw = K.call_args(a, "bf16", "rows")
    x = kw.pop("x0")
    kw["beta"] = kw["beta"][..., 0]
    small = x.clone()
    want = ssm.linear_attention_step(*(t[..., 0] for t in args), small, **kw)["y"]
    pool[rows - 1] = x[0]
    got = ssm.linear_attention_step(*(t[..., 0] for t in args), pool, slots=_int([rows - 1]), **kw)["y"]
    assert torch.equal(got, want) and torch.equal(pool[rows - 1], small[0])


def test_streams():
    """Calls in flight on two streams keep to their own; a call uses the current one."""
    ssm = _ssm()
    sets = []
    for i in range(2):
        a = K.inputs(27 + i, "bf16", 1, 4, 1, 64, 64, 900, pace=0.05)
        args, kw = K.call_args(a, "bf16", "tokens")
        sets.append((args, kw, K.on_device(a["dy"], "bf16", "tokens")))

    def step(args, kw, dy):
        f = ssm.linear_attention(*args, **kw, want_state=True, save=True)
        g = ssm.linear_attention_backward(*args, dy, saved=f["saved"], **kw)
        return [f["y"], f["x"], *(g[k] for k in BACKWARD)]

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for i in range(2) for g in got[i] for p, q in zip(g, want[i]))


def test_captured_decode_with_padding_rows():
    """A decode step captured once; rows are padded by writing -1 into their slots."""
    ssm = _ssm()
    a = K.inputs(29, "bf16", 4, 6, 2, 32, 32, 1)
    args, kw = K.call_args(a, "bf16", "rows")
    x = torch.cat([kw.pop("x0"), torch.zeros((2, 6, 32, 32), device=DEV)])
    kw["beta"] = kw["beta"][..., 0]
    tok, slots = [t[..., 0].clone() for t in args], _int([5, 1, 0, 3])
    y = torch.zeros((4, 6, 32), dtype=torch.bfloat16, device=DEV)
    step = lambda x, y: ssm.linear_attention_step(*tok, x, slots=slots, y=y, **kw)  # noqa: E731
    eager_x, eager_y = x.clone(), y.clone()
    step(x.clone(), y.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, y)
    gen = torch.Generator(device=DEV).manual_seed(30)
    for live in ([5, 1, 0, 3], [5, -1, 0, 3], [-1, -1, 2, -1], [4, 1, 0, 2]):
        slots.copy_(_int(live))
        tok[2].copy_(torch.randn(tok[2].shape, generator=gen, device=DEV))
        graph.replay()
        step(eager_x, eager_y)
        torch.cuda.synchronize()
        assert torch.equal(x, eager_x) and torch.equal(y, eager_y)


def test_refusals_name_the_argument():
    ssm = _ssm()
    a = K.inputs(31, "bf16", 2, 4, 2, 16, 16, 20)
    args, kw = K.call_args(a, "bf16", "tokens")
    q, k, v, g = args
    fwd = lambda q=q, k=k, v=v, g=g, **m: ssm.linear_attention(q, k, v, g, **{**kw, **m})  # noqa: E731
    bwd = lambda dy=v, **m: ssm.linear_attention_backward(q, k, v, g, dy, **{**kw, **m})  # noqa: E731
    step = lambda x, **m: ssm.linear_attention_step(q[..., 0], k[..., 0], v[..., 0], g[..., 0], x, **m)  # noqa: E731
    x = kw["x0"]
    for call, m, name in [
        (fwd, dict(q=q.float()), "q"), (fwd, dict(q=q[..., 0]), "q"), (fwd, dict(k=k[:, :1]), "k"), (fwd, dict(v=v[0]), "v"),
        (fwd, dict(g=g.bfloat16()), "g"), (fwd, dict(g=g[:, :2]), "g"), (fwd, dict(beta=g.double()), "beta"),
        (fwd, dict(D=kw["D"][:2]), "D"), (fwd, dict(x0=x[:1]), "x0"), (fwd, dict(x0=1.0), "x0"), (fwd, dict(x_out=x.half()), "x_out"),
        (fwd, dict(offsets=_int([0, 20]), x0=None), "offsets"), (fwd, dict(lengths=[20, 20]), "lengths"), (fwd, dict(y=v[:1]), "y"),
        (fwd, dict(slots=_int([0, 1]), want_state=True), "slots"), (fwd, dict(slots=_int([0, 1]), x_out=x, save=True), "slots"),
        (bwd, dict(dy=v[..., :4]), "dy"), (bwd, dict(dx=x[:1]), "dx"), (bwd, dict(saved=v), "saved"),
        (step, dict(x=None), "x"), (step, dict(x=x[:1]), "x"), (step, dict(x=x, slots=[0, 1]), "slots"),
        (step, dict(x=x, y=v[..., 0].float()), "y"),
    ]:
        with pytest.raises(ValueError, match=f"^{name}"):
            call(**m)
    with pytest.raises(ssm.SSMError):      # fewer heads than groups
        ssm.linear_attention(q[:, :1].expand(2, 3, 16, 20), k[:, :1].expand(2, 3, 16, 20), v, g)
    with pytest.raises(ssm.SSMError):      # too many keys
        wide = torch.zeros((2, 1, 300, 20), dtype=torch.bfloat16, device=DEV)
        ssm.linear_attention(wide, wide, v, g)
    with pytest.raises(ssm.SSMError):      # states of another call
        bwd(saved=torch.empty(256, dtype=torch.uint8, device=DEV))
