"""Linear attention at finite inputs whose products pass float32: masked places that hold
the type's lowest value, products of large numbers that a small one brings back. What the
definition makes of them in 64 bits has to come out wherever its terms' magnitudes add up
to a number of the result's type. Elsewhere it is not compared: a sum in float32 whose
terms add up to more is infinite, or infinity less infinity, by the order of its terms
(such as the gradient of a masked value, over keys that each have the lowest number).

Tolerances are those of tests/linear_cases.py: roundings against sums of magnitudes, in
which a masked place counts as zero."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import linear_cases as K
from tests.test_gpu_linear import BACKWARD, FORWARD, _f32, _int, _np, _ssm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LARGEST = {"f32": float(np.finfo(np.float32).max), "bf16": 2.0 ** 128 - 2.0 ** 120, "f16": 65504.0}


def compare(a, name, order="tokens", offsets=None, skip_y=(), skip=("dbeta",), at=()):
    """Forward and backward against the oracle; of the steps `at`, the outputs named in `skip` (and y at
    `skip_y`) are left out, and so is what the result's type cannot hold."""
    ssm = _ssm()
    Bsz, _, _, L = a["v"].shape
    spans = S.dense_spans(Bsz, L) if offsets is None else S.packed_spans(offsets)
    args, kw = K.call_args(a, name, order)
    if offsets is not None:
        kw["offsets"] = _int(offsets)
    f = ssm.linear_attention(*args, **kw, want_state=True, save=True)
    g = ssm.linear_attention_backward(*args, K.on_device(a["dy"], name, order), dx=_f32(a["dx"]), saved=f["saved"], **kw)
    torch.cuda.synchronize()
    for got, of, names in ((f, K.forward, FORWARD), (g, K.backward, BACKWARD)):
        want, mag = of(a, spans), of(a, spans, True)
        for n, w in want.items():
            kind = name if n in ("y", "dq", "dk", "dv") else "f32"
            w[mag[n] > 0.9 * LARGEST[kind]] = np.nan
            if n in skip:
                w[..., list(at)] = np.nan
            if n == "y":
                w[..., list(skip_y)] = np.nan
        K.assert_all({n: _np(got[n]) for n in names if got[n] is not None}, want, mag, a, name, spans)


def hide(a, name, what, at, where="lowest"):
    """The masked places `at` of q, k or v: the lowest number of the type."""
    for n in what:
        a[n][..., list(at)] = K.rounded(-LARGEST[name], name) if where == "lowest" else where


SIZES = [(1, 4, 2, 32, 40, 150), (2, 2, 1, 128, 64, 130), (1, 2, 1, 250, 100, 70), (1, 1, 1, 20, 33, 700)]
AT = (5, 20, 21, 31, 32, 64, 69)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("what,zero", [("k", "v"), ("k", "beta"), ("v", "beta"), ("v", "k"), ("kv", "beta"), ("qkv", "beta")])
def test_masked_keys_and_values(name, size, what, zero):
    """A step that adds nothing to the state, by its weight or by what it is paired with."""
    a = K.inputs(41, name, *size, skip=False)
    hide(a, name, what, AT)
    a[zero][..., list(AT)] = 0.0
    a["dy"][..., list(AT)] = 0.0        # nobody reads what a masked step gives
    compare(a, name, skip_y=AT if "q" in what else (), at=AT)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("what,zero", [("k", "v"), ("k", "beta"), ("v", "beta")])
def test_masked_places_that_are_read(name, what, zero):
    """The masked steps' own results count: they are the state's, as it was before."""
    a = K.inputs(42, name, 1, 4, 2, 64, 48, 150, skip=False)
    hide(a, name, what, AT)
    a[zero][..., list(AT)] = 0.0
    compare(a, name, at=AT)


@pytest.mark.parametrize("size", SIZES)
def test_small_numbers_beside_masked_ones_in_float16(size):
    """Keys and values of 3e-3 beside the lowest ones, which weigh nothing: the weights of pairs keep their bits."""
    a = K.inputs(50, "f16", *size, skip=False)
    for n in "kv":
        a[n] = K.rounded(a[n] * 3e-3, "f16")
    a["x0"] = K.rounded(a["x0"] * 1e-5, "f32")
    hide(a, "f16", "kv", AT)
    a["beta"][..., list(AT)] = 0.0
    a["dy"][..., list(AT)] = 0.0
    ssm, spans = _ssm(), S.dense_spans(size[0], size[5])
    args, kw = K.call_args(a, "f16", "tokens")
    g = ssm.linear_attention_backward(*args, K.on_device(a["dy"], "f16", "tokens"), dx=_f32(a["dx"]), **kw)
    want, mag = K.backward(a, spans), K.backward(a, spans, True)
    K.assert_all({n: _np(g[n]) for n in ("dq", "dk", "dv")}, want, mag, a, "f16", spans)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["rows", "mixed"])
def test_masked_places_in_other_orders(name, order):
    a = K.inputs(43, name, 1, 2, 1, 40, 40, 150, skip=False)
    hide(a, name, "kv", AT)
    a["beta"][..., list(AT)] = 0.0
    a["dy"][..., list(AT)] = 0.0
    compare(a, name, order, at=AT)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_masked_places_of_packed_and_cut_sequences(name):
    a = K.inputs(44, name, 1, 1, 1, 32, 48, 900, S=3, skip=False, pace=0.03)
    at = (*AT, 300, 420, 555, 600, 899)
    hide(a, name, "kv", at)
    a["beta"][..., list(at)] = 0.0
    a["dy"][..., list(at)] = 0.0
    compare(a, name, offsets=[0, 290, 610, 900], at=at)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_a_reset_behind_a_masked_place(name):
    """What a masked step put into the state is gone behind a reset (packed documents that a decay of zero parts)."""
    a = K.inputs(45, name, 1, 2, 1, 32, 32, 150, skip=False, beta=False)
    at = (10, 63, 90)
    hide(a, name, "k", at)
    a["v"][..., list(at)] = K.rounded(a["v"][..., list(at)] * 0.01, name)
    a["dy"][..., list(at)] = 0.0
    a["g"][..., [t + 1 for t in at]] = -np.inf
    compare(a, name, skip_y=at, skip=(), at=at)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [dict(k=1e30, q=1e10, v=1e-30), dict(k=1e20, q=1e20, v=1e-32, dy=1e-4),
                                   dict(v=3e37, dy=20.0, k=1e-3, beta=1e-4), dict(k=3e37, v=1e-36, dy=1e3)])
def test_products_that_come_back(name, sizes):
    """q . k (or dy . v) is beyond float32, the results are not.  (dy . v stays above the smallest normal number, 2^-126:
    below it bfloat16's weights of dq and dk have a half step of 2^-134, whatever their size.)"""
    a = K.inputs(46, name, 1, 2, 1, 48, 48, 140, skip=False)
    at = [3, 40, 41, 100]
    for n, s in sizes.items():
        a[n][..., at] = K.rounded(a[n][..., at] * s, "f32" if n == "beta" else name)
    a["x0"] = a["dx"] = None
    if "k" in sizes:
        a["g"][..., [t + 1 for t in at]] = -np.inf      # large keys meet the products of their own step alone
    compare(a, name)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_large_numbers_whose_products_fit(name):
    """Queries and keys of 1e5, values and gradients of 1e10 throughout, as of a scaled loss."""
    a = K.inputs(49, name, 1, 4, 2, 64, 48, 150, skip=False)
    for n, s in dict(q=1e5, k=1e5, v=1e10, dy=1e10).items():
        a[n] = K.rounded(a[n] * s, name)
    a["x0"], a["dx"] = K.rounded(a["x0"] * 1e15, "f32"), K.rounded(a["dx"] * 1e15, "f32")
    compare(a, name, skip=())


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("beta", [0.0, 1.0, 2.5])
def test_step_with_a_masked_key(name, beta):
    """One token whose key or value (or query) is the lowest number and whose other one (state) is zero."""
    ssm = _ssm()
    a = K.inputs(47, name, 2, 4, 2, 32, 40, 1, skip=False)
    a["beta"][:] = beta
    for what, zero in (("k", ("v",)), ("v", ("k",)), ("q", ("x0", "v"))):
        b = {n: v.copy() if isinstance(v, np.ndarray) else v for n, v in a.items()}
        hide(b, name, what, (0,))
        for n in zero:
            b[n][:] = 0.0
        b["scale"] = 3.0 if what == "q" else b["scale"]
        spans = S.dense_spans(2, 1)
        args, kw = K.call_args(b, name, "rows")
        x = kw.pop("x0")
        kw["beta"] = kw["beta"][..., 0]
        y = ssm.linear_attention_step(*(t[..., 0] for t in args), x, **kw)["y"]
        K.assert_all(dict(y=_np(y)[..., None], x=_np(x)), K.forward(b, spans), K.forward(b, spans, True), b, name, spans)


def test_float16_with_states_near_float32s_end():
    """States of up to 3e38 as operands of float16: results that a small scale brings back."""
    for L in (1, 70):
        a = K.inputs(48, "f16", 1, 2, 1, 32, 32, L, skip=False, scale=2.0 ** -110, pace=0.01)
        a["q"] = K.rounded(a["q"] * 1e-3, "f16")
        a["x0"] = K.rounded(a["x0"] / np.abs(a["x0"]).max() * 2.9e38, "f32")
        a["dx"] = K.rounded(a["dx"] * 1e-36, "f32")
        compare(a, "f16", skip=("dq",), at=range(L))


def forward_alone(a, name):
    ssm = _ssm()
    Bsz, H, P, L = a["v"].shape
    G, N = a["q"].shape[1:3]
    assert ssm.linear_bytes(ssm.OP_LINEAR_ATTENTION, K.torch_type(name), Bsz, H, N, P, G, L) > 0      # cut
    spans = S.dense_spans(Bsz, L)
    args, kw = K.call_args(a, name, "tokens")
    f = ssm.linear_attention(*args, **kw, want_state=True)
    K.assert_all({n: _np(f[n]) for n in FORWARD}, K.forward(a, spans), K.forward(a, spans, True), a, name, spans)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [40, 64, 200])
def test_growth_over_pieces(name, N):
    """A cut sequence that grows by more than float32 over a piece, before anything is in its state: what is zero stays
    zero, keys that the kernel pads with among it."""
    a = K.inputs(61, name, 1, 1, 1, N, 24, 1700, carry=False)
    a["g"][..., :1300] = K.rounded((3.5 if name == "f16" else 38.0) / 64, "f32")     # the most that products take
    a["k"][..., :1300] = 0.0
    forward_alone(a, name)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_growth_and_decay_within_a_piece(name):
    """Every piece of 512 steps grows by e^100 and falls by as much, as its states do, from 1e-35 and back."""
    a = K.inputs(62, name, 1, 64, 4, 16, 8, 4096, beta=False)
    a["g"][:] = K.rounded(np.where(np.arange(4096) % 512 < 256, 1.0, -1.0) * 100.0 / 256, "f32")
    a["x0"] = K.rounded(a["x0"] * 1e-35, "f32")
    a["k"][:] = 0.0
    forward_alone(a, name)
