"""The selective operators on the GPU against the float64 oracle: types, storage
orders, head groups, odd sizes, ragged and packed sequences, states and slots,
gradients, single tokens, refusals, streams and captured graphs.

Tolerances count roundings: half a step of the output's type, and half steps
of float32 relative to the sum of magnitudes (tests/selective_cases.py)."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import selective_cases as K

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"


def _ssm():
    from structured_state_space_amd import ssm
    return ssm


def _f32(a):
    return None if a is None else torch.from_numpy(np.asarray(a)).float().to(DEV)


def _np(t):
    return t.detach().double().cpu().numpy()


def _int(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def _sentinel(shape, name, order, value=7.0):
    t = K.on_device(np.full(shape, value), name, order)
    t[...] = value
    return t


# ------------------------------------------------------------- convolution ----

def _conv_args(a, name, order):
    state = None if a["state"] is None else torch.from_numpy(a["state"]).to(K.torch_type(name)).to(DEV)
    return K.on_device(a["u"], name, order), _f32(a["w"]), _f32(a["bias"]), state


def _check_conv(a, name, order, act, spans, **kw):
    ssm = _ssm()
    u, w, b, state = _conv_args(a, name, order)
    W = a["w"].shape[1]
    y = _sentinel(a["u"].shape, name, order)
    out = ssm.causal_conv(u, w, b, silu=act, state=state, want_state=W > 1, y=y, **kw)
    want, last = S.conv(a["u"], a["w"], a["bias"], act, a["state"], spans)
    mag = S.conv(np.abs(a["u"]), np.abs(a["w"]), None if a["bias"] is None else np.abs(a["bias"]), False,
                 None if a["state"] is None else np.abs(a["state"]), spans)[0]
    # W multiply-adds; silu's slope is at most 1.1 and its own error a few steps of the value
    K.assert_near(_np(out["y"]), want, mag, name, 2 * W + 16, "y")
    assert (_np(out["y"])[np.isnan(want)] == 7.0).all(), "a step outside every sequence was written"
    if W > 1:
        assert np.array_equal(_np(out["state"]), last)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["rows", "tokens", "sliced", "mixed"])
@pytest.mark.parametrize("Bsz,H,L,W,act,bias,state", [
    (1, 1, 1, 4, True, True, True),
    (2, 3, 2, 4, True, True, True),        # shorter than the window
    (2, 67, 37, 4, True, True, False),
    (1, 130, 700, 3, False, True, True),   # several workgroups along the steps
    (3, 8, 129, 2, True, False, True),
    (2, 515, 33, 1, True, True, False),
    (1, 9, 1025, 4, False, False, True),
])
def test_conv(name, order, Bsz, H, L, W, act, bias, state):
    a = K.conv_inputs(Bsz + H + L, name, Bsz, H, L, W, bias, state)
    _check_conv(a, name, order, act, S.dense_spans(Bsz, L))


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("H", [8, 9])
def test_conv_long_walks(name, H):
    # enough rows that a thread walks 64 steps and then part of the next 64
    a = K.conv_inputs(45, name, 1030, H, 107, 4, state=True)
    _check_conv(a, name, "tokens", True, S.dense_spans(1030, 107))
    _check_conv_backward(a, name, "tokens", True, S.dense_spans(1030, 107))


@pytest.mark.parametrize("name,order", [("bf16", "tokens"), ("f32", "rows"), ("f16", "mixed")])
def test_conv_packed_and_ragged(name, order):
    offs = [3, 3, 4, 40, 42, 42, 300, 301]   # empty ones, one step, shorter than the window; steps on both sides in none
    a = K.conv_inputs(5, name, 1, 37, 310, 4, state=True, S_=7)
    _check_conv(a, name, order, True, S.packed_spans(offs), offsets=_int(offs))
    lens = [0, 1, 70, 33]
    a = K.conv_inputs(6, name, 4, 37, 70, 4, state=True)
    _check_conv(a, name, order, True, S.dense_spans(4, 70, lens), lengths=_int(lens))


def test_conv_ignores_what_no_sequence_covers():
    a = K.conv_inputs(7, "f32", 1, 20, 64, 4)
    spans = S.packed_spans([5, 20, 50])
    for order in ("rows", "tokens"):
        u, w, b, _ = _conv_args(a, "f32", order)
        u[:, :, :5] = float("nan")
        u[:, :, 50:] = float("inf")
        out = _ssm().causal_conv(u, w, b, silu=True, offsets=_int([5, 20, 50]), want_state=True)
        want, last = S.conv(a["u"], a["w"], a["bias"], True, None, spans)
        K.assert_near(_np(out["y"]), want, np.abs(a["u"]).max() * 4 * np.ones_like(want), "f32", 32, "y")
        assert np.array_equal(_np(out["state"]), last)


def test_conv_slots_and_state_in_place():
    ssm = _ssm()
    a = K.conv_inputs(8, "bf16", 4, 19, 40, 4)
    rng = np.random.default_rng(9)
    pool = K.rounded(rng.standard_normal((6, 19, 3)), "bf16")
    slots = [4, -1, 0, 9]
    for order in ("rows", "tokens"):
        u, w, b, _ = _conv_args(a, "bf16", order)
        state = torch.from_numpy(pool).to(torch.bfloat16).to(DEV)
        y = _sentinel(a["u"].shape, "bf16", order)
        ssm.causal_conv(u, w, b, state=state, state_out=state, slots=_int(slots), y=y)
        after, got = pool.copy(), _np(y)
        for i, s in enumerate(slots):
            if 0 <= s < 6:
                want, last = S.conv(a["u"][i:i + 1], a["w"], a["bias"], False, pool[s:s + 1], S.dense_spans(1, 40))
                K.assert_near(got[i:i + 1], want, 20 * np.ones_like(want), "bf16", 32, "y")
                after[s] = last[0]
            else:
                assert (got[i] == 7.0).all()
        assert np.array_equal(_np(state), after)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["rows", "tokens", "mixed"])
@pytest.mark.parametrize("Bsz,H,L,W,act,bias,state", [
    (1, 1, 1, 4, True, True, True),
    (2, 3, 2, 4, True, True, True),
    (2, 67, 45, 4, True, True, False),
    (1, 20, 2100, 3, True, True, True),   # several workgroups along the steps
    (3, 65, 129, 2, False, False, True),
    (2, 130, 33, 1, True, True, False),
])
def test_conv_backward(name, order, Bsz, H, L, W, act, bias, state):
    a = K.conv_inputs(Bsz + H + L, name, Bsz, H, L, W, bias, state)
    _check_conv_backward(a, name, order, act, S.dense_spans(Bsz, L))


def _check_conv_backward(a, name, order, act, spans, **kw):
    ssm = _ssm()
    rng = np.random.default_rng(10)
    W, n = a["w"].shape[1], len(spans)
    dy = K.rounded(rng.standard_normal(a["u"].shape), name)
    dlast = K.rounded(rng.standard_normal((n, a["w"].shape[0], W - 1)), "f32") if W > 1 else None
    u, w, b, state = _conv_args(a, name, order)
    args = dict(silu=act, state=state, dstate=_f32(dlast), want_dstate=W > 1, **kw)
    out = ssm.causal_conv_backward(u, w, K.on_device(dy, name, order), b, **args)
    want = S.conv_grad(a["u"], a["w"], a["bias"], act, a["state"], dy, dlast, spans)
    mag = S.conv_grad(a["u"], a["w"], a["bias"], act, a["state"], dy, dlast, spans, mag=True)
    # the slope's argument carries 2 W roundings of |w||u|, a slope's change is below
    # half the argument's; then W or, for the parameters, at most 66 sums in float32 (64 of a walk, and the walks)
    rnd = 16 * W + 160
    amp = 1.0 + np.abs(a["w"]).sum(1).max() * np.abs(a["u"]).max()
    K.assert_near(_np(out["du"]), want["du"], amp * mag["du"], name, rnd, "du")
    K.assert_near(_np(out["dweight"]), want["dweight"], amp * mag["dweight"], "f32", rnd, "dweight")
    if b is not None:
        K.assert_near(_np(out["dbias"]), want["dbias"], amp * mag["dbias"], "f32", rnd, "dbias")
    else:
        assert out["dbias"] is None
    if W > 1:
        K.assert_near(_np(out["dstate"]), want["dstate"], amp * mag["dstate"], "f32", rnd, "dstate")
    again = ssm.causal_conv_backward(u, w, K.on_device(dy, name, order), b, **args)
    for k in out:
        assert out[k] is None or torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("name,order", [("bf16", "tokens"), ("f32", "rows"), ("f16", "mixed")])
def test_conv_backward_packed_and_ragged(name, order):
    offs = [3, 3, 4, 40, 42, 42, 300, 301]
    a = K.conv_inputs(11, name, 1, 37, 310, 4, state=True, S_=7)
    _check_conv_backward(a, name, order, True, S.packed_spans(offs), offsets=_int(offs))
    lens = [0, 1, 70, 33]
    a = K.conv_inputs(12, name, 4, 37, 70, 4, state=True)
    _check_conv_backward(a, name, order, True, S.dense_spans(4, 70, lens), lengths=_int(lens))


# -------------------------------------------------------------------- scan ----

def _scan_args(a, name, order):
    dev = lambda v: None if v is None else K.on_device(v, name, order)  # noqa: E731
    return ([dev(a["u"]), dev(a["delta"]), _f32(a["A"]), dev(a["B"]), dev(a["C"])],
            dict(D=_f32(a["D"]), z=dev(a["z"]), delta_bias=_f32(a["bias"]), softplus=a["soft"], x0=_f32(a["x0"])))


def _check_scan(a, name, order, spans, **kw):
    ssm = _ssm()
    args, more = _scan_args(a, name, order)
    y = _sentinel(a["u"].shape, name, order)
    out = ssm.selective_scan(*args, **more, want_state=True, y=y, **kw)
    want, last, _ = K.oracle_scan(a, spans)
    mag, mlast, _ = K.oracle_scan(a, spans, mag=True)
    rnd = K.steps_bound(max(e - b for _, b, e in spans), a["A"].shape[1])
    K.assert_near(_np(out["y"]), want, mag, name, rnd, "y")
    assert (_np(out["y"])[np.isnan(want)] == 7.0).all(), "a step outside every sequence was written"
    K.assert_near(_np(out["x"]), last, mlast, "f32", rnd, "final state")
    # the saving form gives the same bits
    also = ssm.selective_scan(*args, **more, want_state=True, save=True, **kw)
    there = ~torch.isnan(torch.from_numpy(want)).to(DEV)
    assert torch.equal(also["y"][there], out["y"][there]) and torch.equal(also["x"], out["x"])


SCANS = [
    # Bsz, H, L, N, G, gate, skip, bias, soft, state
    (1, 1, 1, 1, 1, True, True, True, True, True),
    (2, 3, 5, 16, 1, True, True, True, True, False),
    (2, 64, 32, 16, 1, False, True, True, True, True),
    (2, 67, 97, 16, 1, True, True, True, True, True),
    (1, 6, 700, 16, 2, True, False, True, True, True),      # chunks
    (1, 130, 333, 8, 2, False, False, False, True, False),  # chunks, two blocks of channels per group
    (3, 12, 70, 3, 4, True, True, False, False, True),
    (2, 20, 50, 24, 1, True, True, True, True, True),       # two blocks of states
    (1, 9, 150, 40, 3, True, True, True, True, True),       # four blocks, the third half full
    (2, 33, 66, 64, 1, True, True, True, False, True),
    (2, 10, 33, 33, 5, True, True, True, True, True),       # groups of fewer channels than a vector, 33 states
    (1, 66, 64, 47, 1, True, True, True, True, False),      # two channels in the second block, whole tiles
    (1, 8, 31, 17, 8, False, True, True, True, True),       # a group per channel
]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["rows", "tokens", "sliced", "mixed"])
@pytest.mark.parametrize("case", SCANS, ids=lambda c: "-".join(map(str, c[:5])))
def test_scan(name, order, case):
    Bsz, H, L, N, G, *flags = case
    a = K.scan_inputs(sum(case[:5]), name, Bsz, H, L, N, G, *flags)
    _check_scan(a, name, order, S.dense_spans(Bsz, L))


OFFSETS = [3, 3, 4, 40, 42, 42, 300, 301, 333]
LENGTHS = [0, 1, 70, 33]


@pytest.mark.parametrize("name,order,N", [("bf16", "tokens", 16), ("f32", "rows", 16), ("f16", "mixed", 20)])
def test_scan_packed_and_ragged(name, order, N):
    a = K.scan_inputs(13, name, 1, 6, 340, N, 2, state=True, S_=8)
    _check_scan(a, name, order, S.packed_spans(OFFSETS), offsets=_int(OFFSETS))
    a = K.scan_inputs(14, name, 4, 6, 70, N, 2, state=True)
    _check_scan(a, name, order, S.dense_spans(4, 70, LENGTHS), lengths=_int(LENGTHS))
    # ragged and long enough for chunks
    a = K.scan_inputs(15, name, 3, 5, 400, N, 1, state=True)
    _check_scan(a, name, order, S.dense_spans(3, 400, [400, 0, 129]), lengths=_int([400, 0, 129]))


def test_scan_many_packed_sequences():
    # more than one wave's worth of sequences for the search of a work item
    rng = np.random.default_rng(16)
    cuts = np.sort(rng.integers(0, 900, 150))
    offs = [0] + [int(v) for v in cuts] + [900]
    a = K.scan_inputs(17, "f32", 1, 3, 900, 4, state=True, S_=len(offs) - 1)
    _check_scan(a, "f32", "tokens", S.packed_spans(offs), offsets=_int(offs))


def test_scan_ignores_what_no_sequence_covers():
    a = K.scan_inputs(18, "f32", 1, 6, 200, 16)
    offs = [7, 60, 60, 171]
    for order in ("rows", "tokens"):
        args, more = _scan_args(a, "f32", order)
        for t in (args[0], args[1], args[3], args[4], more["z"]):
            t[..., :7] = float("nan")
            t[..., 171:] = float("inf")
        out = _ssm().selective_scan(*args, **more, want_state=True, offsets=_int(offs))
        spans = S.packed_spans(offs)
        want, last, _ = K.oracle_scan(a, spans)
        mag, mlast, _ = K.oracle_scan(a, spans, mag=True)
        K.assert_near(_np(out["y"]), want, mag, "f32", K.steps_bound(111, 16), "y")
        K.assert_near(_np(out["x"]), last, mlast, "f32", K.steps_bound(111, 16), "x")


def test_scan_extreme_values():
    # delta of the type's lowest value or -inf: a step of length zero leaves the state as it is
    a = K.scan_inputs(19, "bf16", 1, 5, 40, 16, state=True)
    a["delta"][0, :, 10:14] = -np.inf
    a["delta"][0, :, 20] = float(torch.finfo(torch.bfloat16).min)
    a["delta"][0, 0, 30] = 50.0           # softplus beyond its threshold: a full decay
    _check_scan(a, "bf16", "tokens", S.dense_spans(1, 40))
    # a NaN input reaches its own channel from its step on and no other
    args, more = _scan_args(a, "bf16", "rows")
    ref = _ssm().selective_scan(*args, **more)["y"].clone()
    args[0][0, 2, 25] = float("nan")
    y = _ssm().selective_scan(*args, **more)["y"]
    assert torch.isnan(y[0, 2, 25:]).all()
    ref[0, 2, 25:] = y[0, 2, 25:] = 0
    assert torch.equal(y, ref)


def test_scan_of_huge_steps():
    # a chunk's sum of dt passes float32's range: full decays, and nothing else
    a = K.scan_inputs(52, "f32", 1, 5, 700, 3, gate=False, soft=False, bias=False, state=True)
    a["delta"] = K.rounded(np.full_like(a["delta"], 1e37), "f32")
    a["u"] = K.rounded(a["u"] * 1e-36, "f32")
    spans = S.dense_spans(1, 700)
    for order in ("rows", "tokens"):
        args, more = _scan_args(a, "f32", order)
        out = _ssm().selective_scan(*args, **more, want_state=True)
        want, last, _ = K.oracle_scan(a, spans)
        mag, mlast, _ = K.oracle_scan(a, spans, mag=True)
        K.assert_near(_np(out["y"]), want, mag, "f32", K.steps_bound(1, 3), "y")
        K.assert_near(_np(out["x"]), last, mlast, "f32", K.steps_bound(1, 3), "x")


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_scan_backward_extreme_values(name):
    # steps of length zero (delta -inf or the type's lowest value) hand gradients on
    # and have none of their own; a step past softplus's threshold has slope one
    a = K.scan_inputs(51, name, 2, 5, 70, 16, state=True)
    a["delta"][0, :, 10:14] = -np.inf
    a["delta"][:, 1, 30:66] = float(torch.finfo(K.torch_type(name)).min)
    a["delta"][1, 0, 40] = 50.0
    with np.errstate(over="ignore"):
        _check_scan_backward(a, name, "tokens", S.dense_spans(2, 70))


def test_scan_slots_and_state_in_place():
    ssm = _ssm()
    a = K.scan_inputs(20, "f32", 4, 6, 150, 16)
    pool = K.rounded(np.random.default_rng(21).standard_normal((6, 6, 16)), "f32")
    slots = [4, -1, 0, 9]
    for order in ("rows", "tokens"):   # 150 steps of few channels: chunks
        args, more = _scan_args(a, "f32", order)
        x = _f32(pool)
        y = _sentinel(a["u"].shape, "f32", order)
        more["x0"] = x
        ssm.selective_scan(*args, **more, x_out=x, slots=_int(slots), y=y)
        after, got = pool.copy(), _np(y)
        for i, s in enumerate(slots):
            if 0 <= s < 6:
                one = {k: (v[i:i + 1] if k in ("u", "delta", "z", "B", "C") else v) for k, v in a.items()}
                one["x0"] = pool[s:s + 1]
                want, last, _ = K.oracle_scan(one, S.dense_spans(1, 150))
                mag, mlast, _ = K.oracle_scan(one, S.dense_spans(1, 150), mag=True)
                K.assert_near(got[i:i + 1], want, mag, "f32", K.steps_bound(150, 16), "y")
                K.assert_near(_np(x)[s:s + 1], last, mlast, "f32", K.steps_bound(150, 16), "x")
                after[s] = _np(x)[s]
            else:
                assert (got[i] == 7.0).all()
        assert np.array_equal(_np(x), after)


def _check_scan_backward(a, name, order, spans, dlast=True, **kw):
    ssm = _ssm()
    rng = np.random.default_rng(22)
    H, N = a["A"].shape
    dy = K.rounded(rng.standard_normal(a["u"].shape), name)
    dl = K.rounded(rng.standard_normal((len(spans), H, N)), "f32") if dlast else None
    args, more = _scan_args(a, name, order)
    saved = ssm.selective_scan(*args, **more, save=True, **kw)["saved"]
    dyt = K.on_device(dy, name, order)
    out = ssm.selective_scan_backward(*args, dyt, **more, dx=_f32(dl), saved=saved, **kw)
    want = K.oracle_scan_grad(a, dy, dl, spans)
    mag = K.oracle_scan_grad(a, dy, dl, spans, mag=True)
    rnd = 2 * K.steps_bound(max(max(e - b for _, b, e in spans), 1), N)
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        if out[k] is not None:
            K.assert_near(_np(out[k]), want[k], mag[k], name, rnd, k)
            assert (_np(out[k])[np.isnan(want[k])] == 0).all(), k
    for k in ("dA", "dD", "ddelta_bias", "dx0"):
        if out[k] is not None:
            K.assert_near(_np(out[k]), want[k], mag[k], "f32", rnd, k)
    given = dict(dz=a["z"], dD=a["D"], ddelta_bias=a["bias"], dx0=a["x0"])
    for k, v in given.items():
        assert (out[k] is None) == (v is None), k
    # without the saved states, and a second time: the same bits
    for s in (None, saved):
        again = ssm.selective_scan_backward(*args, dyt, **more, dx=_f32(dl), saved=s, **kw)
        for k in out:
            assert out[k] is None or torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["rows", "tokens", "mixed"])
@pytest.mark.parametrize("case", SCANS, ids=lambda c: "-".join(map(str, c[:5])))
def test_scan_backward(name, order, case):
    Bsz, H, L, N, G, *flags = case
    a = K.scan_inputs(sum(case[:5]), name, Bsz, H, L, N, G, *flags)
    _check_scan_backward(a, name, order, S.dense_spans(Bsz, L), dlast=N != 8)


@pytest.mark.parametrize("name,order,N", [("bf16", "tokens", 16), ("f32", "rows", 16), ("f16", "mixed", 20)])
def test_scan_backward_packed_and_ragged(name, order, N):
    a = K.scan_inputs(23, name, 1, 6, 340, N, 2, state=True, S_=8)
    _check_scan_backward(a, name, order, S.packed_spans(OFFSETS), offsets=_int(OFFSETS))
    a = K.scan_inputs(24, name, 4, 6, 70, N, 2, state=True)
    _check_scan_backward(a, name, order, S.dense_spans(4, 70, LENGTHS), lengths=_int(LENGTHS))


def test_backward_ignores_what_no_sequence_covers():
    ssm = _ssm()
    offs = [7, 60, 60, 171]
    a = K.scan_inputs(25, "f32", 1, 6, 200, 16)
    dy = K.rounded(np.random.default_rng(26).standard_normal(a["u"].shape), "f32")
    ref = None
    for poison in (0.0, float("nan")):
        args, more = _scan_args(a, "f32", "tokens")
        d = K.on_device(dy, "f32", "tokens")
        for t in (args[0], args[1], args[3], args[4], more["z"], d):
            t[..., :7] = poison
            t[..., 171:] = poison
        out = ssm.selective_scan_backward(*args, d, **more, offsets=_int(offs))
        conv = ssm.causal_conv_backward(args[0], torch.ones((6, 4), device=DEV), d, silu=True, offsets=_int(offs))
        out = [v for v in (*out.values(), conv["du"], conv["dweight"]) if v is not None]
        if ref is None:
            ref = out
        else:
            assert all(torch.equal(p, q) for p, q in zip(ref, out))


def test_scan_gradient_matches_differences_of_the_kernel():
    # float32: one direction through every input, a step of 2^-7 of it, against the gradients' product with it
    ssm = _ssm()
    a = K.scan_inputs(27, "f32", 1, 8, 60, 16, state=True)
    rng = np.random.default_rng(28)
    args, more = _scan_args(a, "f32", "tokens")
    names = ["u", "delta", "A", "B", "C", "D", "z", "delta_bias", "x0"]
    vals = dict(zip(names[:5], args), **{k: more[k] for k in names[5:]})
    dirs = {k: torch.from_numpy(rng.standard_normal(v.shape)).float().to(DEV) * (0.1 if k in ("A", "delta_bias") else 1)
            for k, v in vals.items()}
    dy = torch.from_numpy(rng.standard_normal(a["u"].shape)).float().to(DEV)

    def loss(step):
        v = {k: t + step * dirs[k] for k, t in vals.items()}
        out = ssm.selective_scan(v["u"], v["delta"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"],
                                 delta_bias=v["delta_bias"], softplus=True, x0=v["x0"])
        return float((out["y"].double() * dy.double()).sum())

    g = ssm.selective_scan_backward(*args, dy, **more)
    slope = sum(float((g["d" + k].double() * dirs[k].double()).sum()) for k in names)
    e = 2.0 ** -7
    # five-point rule: its error is of fourth order in the step
    diff = (8 * (loss(e) - loss(-e)) - (loss(2 * e) - loss(-2 * e))) / (12 * e)
    assert abs(diff - slope) <= 1e-3 * abs(slope), (diff, slope)


# ----------------------------------------------------------- single tokens ----

@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Bsz,H,N,G,gate", [(1, 1, 1, 1, True), (3, 67, 16, 1, True), (5, 130, 24, 2, False),
                                           (2, 48, 40, 3, True), (2, 9, 64, 1, True), (4100, 64, 7, 1, True),
                                           (4100, 64, 16, 1, False)])
def test_selective_step(name, Bsz, H, N, G, gate):
    ssm = _ssm()
    a = K.scan_inputs(29, name, Bsz, H, 1, N, G, gate, state=True)
    tok = lambda v: None if v is None else torch.from_numpy(v[..., 0]).to(K.torch_type(name)).to(DEV)  # noqa: E731
    wide = torch.cat([tok(a["u"]), tok(a["delta"])], 1)    # rows of a wider projection
    x = _f32(a["x0"])
    out = ssm.selective_step(wide[:, :H], wide[:, H:], _f32(a["A"]), tok(a["B"]), tok(a["C"]), x, D=_f32(a["D"]),
                             z=tok(a["z"]), delta_bias=_f32(a["bias"]), softplus=True)
    spans = S.dense_spans(Bsz, 1)
    want, last, _ = K.oracle_scan(a, spans)
    mag, mlast, _ = K.oracle_scan(a, spans, mag=True)
    K.assert_near(_np(out["y"]), want[..., 0], mag[..., 0], name, K.steps_bound(1, N), "y")
    K.assert_near(_np(out["x"]), last, mlast, "f32", K.steps_bound(1, N), "x")
    assert out["x"] is x


@pytest.mark.parametrize("Bsz,H,N,G", [(3, 130, 16, 2), (2, 12, 24, 4), (300, 1030, 16, 2), (2, 5, 1, 1)])
def test_selective_step_strides(Bsz, H, N, G):
    # B and C with the groups stored last, or one B for all states: what their copies give
    ssm = _ssm()
    g = torch.Generator(device=DEV).manual_seed(53)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()  # noqa: E731
    u, delta, B, C, b1 = r(Bsz, H), r(Bsz, H), r(Bsz, N, G).transpose(1, 2), r(Bsz, N, G).transpose(1, 2), r(Bsz, G, 1)
    A, x = -torch.rand((H, N), generator=g, device=DEV), torch.randn((Bsz, H, N), generator=g, device=DEV)
    for B in (B, b1.expand(Bsz, G, N)):
        got = ssm.selective_step(u, delta, A, B, C, x.clone(), softplus=True)
        want = ssm.selective_step(u, delta, A, B.contiguous(), C.contiguous(), x.clone(), softplus=True)
        assert torch.equal(got["y"], want["y"]) and torch.equal(got["x"], want["x"])


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Bsz,H,W,act,bias", [(1, 1, 4, True, True), (3, 67, 4, True, True), (5, 130, 3, False, False),
                                             (2, 48, 2, True, True), (2, 9, 1, True, True), (300, 1030, 4, True, True)])
def test_conv_step(name, Bsz, H, W, act, bias):
    ssm = _ssm()
    a = K.conv_inputs(30, name, Bsz, H, 1, W, bias, True)
    _, w, b, state = _conv_args(a, name, "rows")
    u = torch.from_numpy(a["u"][..., 0]).to(K.torch_type(name)).to(DEV)
    out = ssm.causal_conv_step(u, w, state, b, silu=act)
    want, last = S.conv(a["u"], a["w"], a["bias"], act, a["state"], S.dense_spans(Bsz, 1))
    K.assert_near(_np(out["y"]), want[..., 0], 30 * np.ones((Bsz, H)), name, 2 * W + 16, "y")
    if W > 1:
        assert np.array_equal(_np(out["state"]), last) and out["state"] is state


def test_step_slots():
    ssm = _ssm()
    rng = np.random.default_rng(31)
    slots = [3, -1, 0, 7, 2**31 - 1, 5]
    a = K.scan_inputs(32, "bf16", 6, 70, 1, 16)
    c = K.conv_inputs(33, "bf16", 6, 70, 1, 4)
    pool, cpool = K.rounded(rng.standard_normal((7, 70, 16)), "f32"), K.rounded(rng.standard_normal((7, 70, 3)), "bf16")
    tok = lambda v: torch.from_numpy(v[..., 0]).bfloat16().to(DEV)  # noqa: E731
    x, st = _f32(pool), torch.from_numpy(cpool).bfloat16().to(DEV)
    y, yc = torch.full((6, 70), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((6, 70), 7.0, dtype=torch.bfloat16, device=DEV)
    ssm.selective_step(tok(a["u"]), tok(a["delta"]), _f32(a["A"]), tok(a["B"]), tok(a["C"]), x, D=_f32(a["D"]),
                       z=tok(a["z"]), delta_bias=_f32(a["bias"]), softplus=True, slots=_int(slots), y=y)
    ssm.causal_conv_step(tok(c["u"]), _f32(c["w"]), st, _f32(c["bias"]), silu=True, slots=_int(slots), y=yc)
    after, cafter = pool.copy(), cpool.copy()
    for i, s in enumerate(slots):
        if not 0 <= s < 7:
            assert (_np(y)[i] == 7).all() and (_np(yc)[i] == 7).all()
            continue
        one = {k: (v[i:i + 1] if k in ("u", "delta", "z", "B", "C") else v) for k, v in a.items()}
        one["x0"] = pool[s:s + 1]
        want, last, _ = K.oracle_scan(one, S.dense_spans(1, 1))
        mag, mlast, _ = K.oracle_scan(one, S.dense_spans(1, 1), mag=True)
        K.assert_near(_np(y)[i:i + 1], want[..., 0], mag[..., 0], "bf16", K.steps_bound(1, 16), "y")
        K.assert_near(_np(x)[s:s + 1], last, mlast, "f32", K.steps_bound(1, 16), "x")
        want, last = S.conv(c["u"][i:i + 1], c["w"], c["bias"], True, cpool[s:s + 1], S.dense_spans(1, 1))
        K.assert_near(_np(yc)[i:i + 1], want[..., 0], 30 * np.ones((1, 70)), "bf16", 32, "y")
        after[s], cafter[s] = _np(x)[s], last[0]
    assert np.array_equal(_np(x), after) and np.array_equal(_np(st), cafter)


# --------------------------------------------------------------- together ----

def _block_weights(H, N, name, seed=34):
    r = np.random.default_rng(seed)
    p = K.conv_inputs(seed, name, 1, H, 1, 4)
    a = K.scan_inputs(seed, name, 1, H, 1, N)
    return dict(w=_f32(p["w"]), cb=_f32(p["bias"]), A=_f32(a["A"]), D=_f32(a["D"]), bias=_f32(a["bias"]),
                proj=torch.from_numpy(r.standard_normal((H, H + 2 * N)) / np.sqrt(H)).float().to(DEV))


def _prefill(P, xz, N, conv, x, name, **kw):
    """A block's sequence mixer over tokens xz [T, 2 H] of packed prompts: convolution, projections, scan."""
    ssm = _ssm()
    H = xz.shape[1] // 2
    u, z = xz[None, :, :H].transpose(1, 2), xz[None, :, H:].transpose(1, 2)
    u = ssm.causal_conv(u, P["w"], P["cb"], silu=True, state=conv, state_out=conv, **kw)["y"]
    dbc = (u[0].t().float() @ P["proj"]).to(xz.dtype)[None]            # [1, T, H + 2 N]
    d, B, C = dbc[..., :H].transpose(1, 2), dbc[..., H:H + N], dbc[..., H + N:]
    return ssm.selective_scan(u, d, P["A"], B.transpose(1, 2)[:, None], C.transpose(1, 2)[:, None], D=P["D"], z=z,
                              delta_bias=P["bias"], softplus=True, x0=x, x_out=x, **kw)["y"][0].t()


def _decode(P, xz, N, conv, x, slots):
    ssm = _ssm()
    H = xz.shape[1] // 2
    u = ssm.causal_conv_step(xz[:, :H], P["w"], conv, P["cb"], silu=True, slots=slots)["y"]
    dbc = (u.float() @ P["proj"]).to(xz.dtype)
    return ssm.selective_step(u, dbc[:, :H], P["A"], dbc[:, None, H:H + N], dbc[:, None, H + N:], x, D=P["D"],
                              z=xz[:, H:], delta_bias=P["bias"], softplus=True, slots=slots)["y"]


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_prompts_then_tokens(name):
    """Packed prompts into a pool of slots, one of them in two pieces, then three
    decode steps: equal to each whole sequence in one call."""
    H, N, pool = 72, 16, 5
    P = _block_weights(H, N, name)
    t = K.torch_type(name)
    g = torch.Generator(device=DEV).manual_seed(35)
    lens, slots = [70, 1, 33], [3, 0, 4]
    xs = [torch.randn((n + 3, 2 * H), generator=g, device=DEV).to(t) for n in lens]
    conv, x = torch.zeros((pool, H, 3), dtype=t, device=DEV), torch.zeros((pool, H, N), device=DEV)
    # first 41 steps of the first prompt by themselves
    first = _prefill(P, xs[0][:41], N, conv, x, name, offsets=_int([0, 41]), slots=_int([3]))
    rest = [xs[0][41:70], xs[1][:1], xs[2][:33]]
    offs = [0, 29, 30, 63]
    y = _prefill(P, torch.cat(rest), N, conv, x, name, offsets=_int(offs), slots=_int(slots))
    got = [[first, y[:29]], [y[29:30]], [y[30:]]]
    for k in range(3):
        yk = _decode(P, torch.stack([v[n + k] for v, n in zip(xs, lens)]), N, conv, x, _int(slots))
        for i in range(3):
            got[i].append(yk[i:i + 1])
    for i, v in enumerate(xs):
        c1, x1 = torch.zeros((1, H, 3), dtype=t, device=DEV), torch.zeros((1, H, N), device=DEV)
        whole = _prefill(P, v, N, c1, x1, name, offsets=_int([0, v.shape[0]]))
        mine = torch.cat(got[i])
        # the same arithmetic but for where a sequence is cut; a projection's rounding may
        # fall to the other side, which moves its consumer by a step of the type
        scale = float(whole.float().abs().max())
        assert float((mine.float() - whole.float()).abs().max()) <= scale * 32 * K.HALF_STEP[name] + scale * 1e-5
        assert torch.equal(conv[slots[i]], c1[0])


def test_training_step_against_differences():
    """Convolution and scan forward and backward together, through a loss."""
    ssm = _ssm()
    H, L, N = 24, 50, 16
    a, c = K.scan_inputs(36, "f32", 2, H, L, N), K.conv_inputs(36, "f32", 2, H, L, 4)
    args, more = _scan_args(a, "f32", "tokens")
    u0, w, cb, _ = _conv_args(c, "f32", "tokens")
    g = torch.Generator(device=DEV).manual_seed(37)
    dy = torch.randn((2, H, L), generator=g, device=DEV)
    du0, dw = torch.randn(u0.shape, generator=g, device=DEV), torch.randn(w.shape, generator=g, device=DEV)

    def loss(e):
        u = ssm.causal_conv(u0 + e * du0, w + e * dw, cb, silu=True)["y"]
        y = ssm.selective_scan(u, *args[1:], **more)["y"]
        return float((y.double() * dy.double()).sum())

    u = ssm.causal_conv(u0, w, cb, silu=True)["y"]
    fwd = ssm.selective_scan(u, *args[1:], **more, save=True)
    gs = ssm.selective_scan_backward(u, *args[1:], dy, **more, saved=fwd["saved"])
    gc = ssm.causal_conv_backward(u0, w, gs["du"], cb, silu=True)
    slope = float((gc["du"].double() * du0).sum() + (gc["dweight"].double() * dw).sum())
    e = 2.0 ** -7
    diff = (8 * (loss(e) - loss(-e)) - (loss(2 * e) - loss(-2 * e))) / (12 * e)
    assert abs(diff - slope) <= 1e-3 * abs(slope), (diff, slope)


def test_broadcast_inputs():
    """Inputs that repeat along the batch, the channels, the states or the steps
    (stride 0) give what their copies give, and so do the gradients."""
    ssm = _ssm()
    Bsz, H, N, L = 3, 12, 16, 70
    g = torch.Generator(device=DEV).manual_seed(46)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()  # noqa: E731
    u, delta, z = r(1, H, L).expand(Bsz, H, L), r(Bsz, 1, L).expand(Bsz, H, L), r(Bsz, H, 1).expand(Bsz, H, L)
    B, C = r(Bsz, 1, 1, L).expand(Bsz, 2, N, L), r(1, 2, N, 1).expand(Bsz, 2, N, L)
    A, dy = -torch.rand((H, N), generator=g, device=DEV), r(Bsz, 1, 1).expand(Bsz, H, L)
    w = torch.randn((H, 4), generator=g, device=DEV)

    def step(f):
        v = [f(t) for t in (u, delta, A, B, C)]
        fw = ssm.selective_scan(*v, z=f(z), softplus=True, want_state=True)
        bw = ssm.selective_scan_backward(*v, f(dy), z=f(z), softplus=True)
        cv = ssm.causal_conv(f(u), w, silu=True)
        cb = ssm.causal_conv_backward(f(delta), w, f(dy), silu=True)
        dw = cb.pop("dweight")
        return [t for d in (fw, bw, cv, cb) for t in d.values() if t is not None], dw

    (got, dw), (want, dw_want) = step(lambda t: t), step(lambda t: t.contiguous())
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    # the two storage orders add a weight's 210 terms d_t u_t in different orders: at
    # most 80 float32 additions in a row on either side (a row's 70 steps and the
    # threads' sums; rows are added in float64), each off by half a step of at most
    # the terms' magnitudes, |d| <= 1.1 |dy|
    most = 1.1 * (dy.double().abs() * delta.double().abs().max()).sum((0, 2))
    assert ((dw.double() - dw_want.double()).abs() <= 2 * 80 * 2.0 ** -24 * most[:, None]).all()
    with pytest.raises(ssm.SSMError):   # an output must not repeat
        ssm.causal_conv(u.contiguous(), w, y=torch.empty((1, H, L), dtype=u.dtype, device=DEV).expand(Bsz, H, L))


def _far(t, stride):
    """`t` [Bsz, ..., L] with batch rows, or its steps if it has one row, `stride` elements apart."""
    moved = t.movedim(-1, 1).contiguous()                          # [Bsz, L, ...]
    apart = list(moved.stride())
    apart[0 if t.shape[0] > 1 else 1] = stride
    n = sum((d - 1) * v for d, v in zip(moved.shape, apart)) + 1
    out = torch.empty(n, dtype=t.dtype, device=DEV).as_strided(moved.shape, apart)
    return out.copy_(moved).movedim(1, -1)


@pytest.mark.parametrize("Bsz,L,stride", [(2, 70, 2**31 + 64), (1, 600, 2**22)])
def test_offsets_past_32_bits(Bsz, L, stride):
    """Rows further apart than 2^31 elements, and steps that end there: what dense
    copies give, bit for bit."""
    ssm = _ssm()
    a = K.scan_inputs(54, "bf16", Bsz, 72, L, 16, state=True)
    c = K.conv_inputs(55, "bf16", Bsz, 72, L, 4, state=True)
    args, more = _scan_args(a, "bf16", "tokens")
    u0, w, cb, state = _conv_args(c, "bf16", "tokens")

    def step(f):
        fw = ssm.selective_scan(f(args[0]), f(args[1]), args[2], *args[3:], **more, want_state=True, y=f(args[0]))
        bw = ssm.selective_scan_backward(f(args[0]), *args[1:], f(args[1]), **more)
        cv = ssm.causal_conv(f(u0), w, cb, silu=True, state=state, want_state=True, y=f(u0))
        cg = ssm.causal_conv_backward(f(u0), w, f(args[1]), cb, silu=True, state=state)
        return [t.contiguous() for d in (fw, bw, cv, cg) for t in d.values() if t is not None]

    for p, q in zip(step(lambda t: _far(t, stride)), step(lambda t: t.clone())):
        assert torch.equal(p, q)


def test_pool_past_32_bits():
    ssm = _ssm()
    H, N = 4096, 16
    rows = 2**31 // (H * N) + 3
    g = torch.Generator(device=DEV).manual_seed(56)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()  # noqa: E731
    x = torch.empty((rows, H, N), device=DEV)
    conv = torch.empty((2**31 // (H * 3) + 3, H, 3), dtype=torch.bfloat16, device=DEV)
    sx, sc = _int([rows - 1, 5]), _int([conv.shape[0] - 1, 5])
    first, cfirst = torch.randn((2, H, N), generator=g, device=DEV), r(2, H, 3)
    x[sx.long()], conv[sc.long()] = first, cfirst
    u, delta, B, C, w = r(2, H), r(2, H), r(2, 1, N), r(2, 1, N), torch.randn((H, 4), generator=g, device=DEV)
    A = -torch.rand((H, N), generator=g, device=DEV)
    for args in ((u, delta, A, B, C), tuple(t if t is A else t[..., None] for t in (u, delta, A, B, C))):
        if args[0].dim() == 2:
            y = ssm.selective_step(*args, x, softplus=True, slots=sx)["y"]
            want = ssm.selective_step(*args, first, softplus=True)
        else:
            y = ssm.selective_scan(*args, softplus=True, x0=x, x_out=x, slots=sx)["y"]
            want = ssm.selective_scan(*args, softplus=True, x0=first, x_out=first)
        assert torch.equal(y, want["y"]) and torch.equal(x[sx.long()], first)
    y = ssm.causal_conv_step(u, w, conv, slots=sc)["y"]
    assert torch.equal(y, ssm.causal_conv_step(u, w, cfirst)["y"]) and torch.equal(conv[sc.long()], cfirst)
    y = ssm.causal_conv(u[..., None], w, state=conv, state_out=conv, slots=sc)["y"]
    assert torch.equal(y, ssm.causal_conv(u[..., None], w, state=cfirst, state_out=cfirst)["y"])
    assert torch.equal(conv[sc.long()], cfirst)


def test_workspace_is_checked():
    ssm = _ssm()
    a = K.scan_inputs(47, "f32", 1, 6, 400, 16)
    args, more = _scan_args(a, "f32", "rows")
    n = ssm.selective_bytes(ssm.OP_SELECTIVE_SCAN, 1, 6, 16, 1, 400)
    assert n > 0
    ref = ssm.selective_scan(*args, **more)["y"]
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2],
                torch.empty(n - 1, dtype=torch.uint8, device=DEV)):
        with pytest.raises(ValueError):
            ssm.selective_scan(*args, **more, workspace=bad)
    with pytest.raises(ssm.SSMError):   # not on a multiple of 256 bytes
        ssm.selective_scan(*args, **more, workspace=torch.empty(n + 4, dtype=torch.uint8, device=DEV)[4:])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert torch.equal(ssm.selective_scan(*args, **more, workspace=ws)["y"], ref)


# ------------------------------------------------------ streams and graphs ----

def test_two_streams_at_once():
    """Calls with workspaces in flight on two streams keep to their own."""
    ssm = _ssm()
    sets = [_scan_args(K.scan_inputs(48 + i, "bf16", 1, 200, 3000, 16), "bf16", "tokens") for i in range(2)]

    def step(args, more):
        f = ssm.selective_scan(*args, **more, want_state=True, save=True)
        b = ssm.selective_scan_backward(*args, args[0], **more, saved=f["saved"])
        c = ssm.causal_conv_backward(args[0], W, args[1], silu=True)
        return [v for d in (f, b, c) for k, v in d.items() if v is not None and k != "saved"]

    W = torch.randn((200, 4), generator=torch.Generator(device=DEV).manual_seed(50), device=DEV)
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for p, q in zip(g, want[i]):
                assert torch.equal(p, q)


def test_on_another_stream():
    ssm = _ssm()
    a = K.scan_inputs(38, "bf16", 1, 40, 500, 16)
    args, more = _scan_args(a, "bf16", "tokens")
    ref = ssm.selective_scan(*args, **more, want_state=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ssm.selective_scan(*args, **more, want_state=True)
        back = ssm.selective_scan_backward(*args, args[0], **more)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(ref["y"], got["y"]) and torch.equal(ref["x"], got["x"])
    assert torch.equal(back["du"], ssm.selective_scan_backward(*args, args[0], **more)["du"])


def test_captured_training_step():
    """Forward and backward of both operators in one graph, replayed with new
    inputs between eager calls: every replay equals the eager result."""
    ssm = _ssm()
    H, L = 40, 300
    a, c = K.scan_inputs(39, "bf16", 2, H, L, 16, state=True), K.conv_inputs(39, "bf16", 2, H, L, 4)
    args, more = _scan_args(a, "bf16", "tokens")
    u0, w, cb, _ = _conv_args(c, "bf16", "tokens")
    dy = K.on_device(K.rounded(np.random.default_rng(40).standard_normal((2, H, L)), "bf16"), "bf16", "tokens")

    def step():
        u = ssm.causal_conv(u0, w, cb, silu=True)["y"]
        f = ssm.selective_scan(u, *args[1:], **more, want_state=True, save=True)
        g = ssm.selective_scan_backward(u, *args[1:], dy, **more, saved=f["saved"])
        k = ssm.causal_conv_backward(u0, w, g["du"], cb, silu=True)
        return [v for v in (f["y"], f["x"], *g.values(), *k.values()) if v is not None]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    g = torch.Generator(device=DEV).manual_seed(41)
    for _ in range(4):
        u0.copy_(torch.randn(u0.shape, generator=g, device=DEV))
        dy.copy_(torch.randn(dy.shape, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        for p, q in zip(got, step()):
            assert torch.equal(p, q)


def test_captured_decode_with_padding_rows():
    """A decode step captured once; the batch shrinks by writing -1 into its slots."""
    ssm = _ssm()
    H, N, rows = 72, 16, 6
    P = _block_weights(H, N, "bf16", 42)
    g = torch.Generator(device=DEV).manual_seed(43)
    conv = torch.randn((rows, H, 3), generator=g, device=DEV).bfloat16()
    x = torch.randn((rows, H, N), generator=g, device=DEV)
    slots, xz = _int([0, 1, 2, 3]), torch.randn((4, 2 * H), generator=g, device=DEV).bfloat16()
    u, y = torch.empty((4, H), dtype=torch.bfloat16, device=DEV), torch.empty((4, H), dtype=torch.bfloat16, device=DEV)
    bc = torch.randn((4, 2, 1, N), generator=g, device=DEV).bfloat16()

    def step(conv, x, u, y):
        ssm.causal_conv_step(xz[:, :H], P["w"], conv, P["cb"], silu=True, slots=slots, y=u)
        ssm.selective_step(u, xz[:, H:], P["A"], bc[:, 0], bc[:, 1], x, D=P["D"], z=xz[:, H:],
                           delta_bias=P["bias"], softplus=True, slots=slots, y=y)

    eager = [v.clone() for v in (conv, x, u, y)]
    graph = torch.cuda.CUDAGraph()
    step(*[v.clone() for v in (conv, x, u, y)])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(conv, x, u, y)
    for s in ([0, 1, 2, 3], [5, -1, 2, 0], [-1, -1, -1, 4], [3, 2, 1, 0]):
        slots.copy_(_int(s))
        xz.copy_(torch.randn(xz.shape, generator=g, device=DEV))
        u.fill_(1.0), y.fill_(1.0), eager[2].fill_(1.0), eager[3].fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        step(*eager)
        for p, q in zip((conv, x, u, y), eager):
            assert torch.equal(p, q)
