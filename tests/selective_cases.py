"""Inputs, tolerances and torch views shared by the selective operators' tests."""
import numpy as np

import oracle.selective_oracle as S

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the smallest subnormal


def torch_type(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def rounded(a, name):
    """float64 values of `a` after rounding to the type."""
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).to(torch_type(name)).double().numpy()


def on_device(a, name, order, dev="cuda:0"):
    """`a` [Bsz, ..., L] as a device tensor of the type, stored in the given order:
    "rows" (steps contiguous), "tokens" (steps first behind the batch), "sliced"
    (tokens, every row a slice of a wider one) or "mixed" (neither the steps nor
    the channels contiguous)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch_type(name)).to(dev)
    if order == "rows":
        return t.contiguous()
    moved = t.movedim(-1, 1)  # [Bsz, L, ...]
    if order == "tokens":
        return moved.contiguous().movedim(1, -1)
    if order == "sliced":
        wide = torch.full((*moved.shape[:-1], moved.shape[-1] + 5), float("nan"), dtype=t.dtype, device=dev)
        wide[..., 3:3 + moved.shape[-1]] = moved
        return wide[..., 3:3 + moved.shape[-1]].movedim(1, -1)
    wide = torch.full((*moved.shape, 2), float("nan"), dtype=t.dtype, device=dev)
    wide[..., 1] = moved
    return wide[..., 1].movedim(1, -1)


def steps_bound(L, N):
    """Float32 roundings that can meet in one value: per step of the recurrence
    the decay (its exponent's two products, the exponential, dt's own handful)
    and one multiply-add, below 16 half steps with |dt A| <= 1, over at most L
    steps there and L back; the sum over N states; a constant number more."""
    return 16 * 2 * L + 2 * N + 64


def assert_near(got, want, mag, name, roundings, what):
    """|got - want| <= half a step of the output's type relative to the value, plus
    `roundings` half steps of float32 relative to the sum of magnitudes `mag`.
    NaN in `want` marks what is not written and not compared."""
    got, want, mag = (np.asarray(v, dtype=np.float64) for v in (got, want, mag))
    assert got.shape == want.shape, (what, got.shape, want.shape)
    there = ~np.isnan(want)
    # the float32 error itself is rounded with the value
    f32 = roundings * 2.0 ** -24 * mag
    tol = HALF_STEP[name] * (np.abs(want) + f32) + f32 + SMALLEST[name]
    bad = there & ~(np.abs(got - want) <= tol)
    if bad.any():
        at = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(there.sum())} off, first at {at}: "
                             f"{got[at]} for {want[at]}, tolerance {tol[at]:.3g}")


def scan_inputs(seed, name, Bsz, H, L, N, G=1, gate=True, skip=True, bias=True, soft=True, state=False, S_=None):
    """Values of the types the device sees, as float64."""
    r = np.random.default_rng(seed)
    act = lambda *s: rounded(r.standard_normal(s), name)  # noqa: E731
    par = lambda v: rounded(v, "f32")  # noqa: E731
    a = dict(u=act(Bsz, H, L), B=act(Bsz, G, N, L), C=act(Bsz, G, N, L))
    a["A"] = par(-np.arange(1, N + 1) * np.exp(0.2 * r.standard_normal((H, N))))
    # dt |A| <= 1: dt up to 1 / (2 N)
    dt = np.exp(r.uniform(np.log(1e-3), np.log(0.1), H)) / max(1, N // 8)
    if soft:
        a["delta"] = rounded(0.5 * r.standard_normal((Bsz, H, L)), name)
        a["bias"] = par(dt + np.log(-np.expm1(-dt))) if bias else None
        if not bias:
            a["delta"] = rounded(a["delta"] - 5.0, name)
    else:
        a["delta"] = rounded(dt[:, None] * np.exp(0.3 * r.standard_normal((Bsz, H, L))), name)
        a["bias"] = par(1e-3 * r.random(H)) if bias else None
    a["D"] = par(r.standard_normal(H)) if skip else None
    a["z"] = act(Bsz, H, L) if gate else None
    a["x0"] = par(r.standard_normal((S_ or Bsz, H, N))) if state else None
    a["soft"] = soft
    return a


def conv_inputs(seed, name, Bsz, H, L, W, bias=True, state=False, S_=None):
    r = np.random.default_rng(seed)
    return dict(u=rounded(r.standard_normal((Bsz, H, L)), name),
                w=rounded(r.standard_normal((H, W)) / np.sqrt(W), "f32"),
                bias=rounded(0.3 * r.standard_normal(H), "f32") if bias else None,
                state=rounded(r.standard_normal((S_ or Bsz, H, W - 1)), name) if state and W > 1 else None)


def oracle_scan(a, spans, mag=False):
    return S.scan(a["u"], a["delta"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], a["soft"], a["x0"], spans, mag)


def oracle_scan_grad(a, dy, dlast, spans, mag=False):
    return S.scan_grad(a["u"], a["delta"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], a["soft"], a["x0"], dy,
                       dlast, spans, mag)
