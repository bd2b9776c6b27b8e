"""Inputs, tolerances and torch views of the linear attention and layer norm tests.

Roundings are counted in half steps of float32, U = 2^-24 relative, against sums of
magnitudes (the oracle with mag=True).  Of linear attention:

    weight of a pair   three sums of log decays, each of at most 17 additions and of
                       at most D, the most that |g| adds up to over 64 steps: 51 D; their
                       exponentials 3 (|argument| + 4), products 4: 54 D + 16
    state              per chunk the decay's factor (16 D + 4) and an addition; so many
                       chunks; 64 kParts + 4 additions of products within one, operands
                       split to 2^-22 or better (4 half steps)
    result             the state's, 3 N + 64 additions more
    gradients          the same walk back, and sums over 64 values and N keys

so that C(chunks, N, D) below bounds them all.  Results of a 16-bit type have one
factor of each product rounded to it (half a step of the type against the magnitudes)
and are rounded themselves.  dg is a difference of running sums over a chunk: its
roundings are relative to the chunk's sums."""
import numpy as np

import oracle.linear_oracle as O
from tests.selective_cases import HALF_STEP, SMALLEST, on_device, rounded, torch_type  # noqa: F401

U = 2.0 ** -24


def inputs(seed, name, Bsz, H, G, N, P, L, S=None, beta=True, skip=True, carry=True, pace=0.2, scale=None):
    """Values of the types the device sees, as float64."""
    r = np.random.default_rng(seed)
    act = lambda *s: rounded(r.standard_normal(s), name)  # noqa: E731
    f = lambda a: rounded(a, "f32")  # noqa: E731
    S = S or Bsz
    return dict(q=act(Bsz, G, N, L), k=act(Bsz, G, N, L), v=act(Bsz, H, P, L),
                g=f(-pace * r.exponential(size=(Bsz, H, L)) * r.random((H, 1))),
                beta=f(r.random((Bsz, H, L)) * 2.0) if beta else None,
                D=f(r.standard_normal(H)) if skip else None,
                scale=float(np.float32(N ** -0.5 if scale is None else scale)),
                x0=f(r.standard_normal((S, H, N, P))) if carry else None,
                dy=act(Bsz, H, P, L), dx=f(r.standard_normal((S, H, N, P))) if carry else None)


def forward(a, spans, mag=False):
    y, x, _ = O.attention(a["q"], a["k"], a["v"], a["g"], a["beta"], a["D"], a["scale"], a["x0"], spans, mag)
    return dict(y=y, x=x)


def backward(a, spans, mag=False):
    return O.attention_grad(a["q"], a["k"], a["v"], a["g"], a["beta"], a["D"], a["scale"], a["x0"], a["dy"], a["dx"],
                            spans, mag)


def roundings(a):
    L, N = a["q"].shape[3], a["q"].shape[2]
    total = np.cumsum(np.abs(np.concatenate([np.zeros((*a["g"].shape[:2], 1)), np.where(np.isinf(a["g"]), 0.0, a["g"])], 2)), 2)
    D = (total[:, :, 64:] - total[:, :, :-64]).max() if L >= 64 else total[:, :, -1].max()
    chunks = 2 * (L // 32 + 2)     # there and back
    return chunks * (16.0 * D + 8.0) + 54.0 * D + 3.0 * N + 3.0 * 64 * 4 + 128.0


def assert_all(got, want, mag, a, name, spans, what=""):
    """Every output of a call against the oracle's, within the counted roundings; and, of the float32
    ones, the norm of the error against that of the result: independent roundings add up to
    their root, with (16 + 4 D + 2 sqrt(64)) half steps a generous count of each element's."""
    count = roundings(a)
    for n, w in want.items():
        if n not in got or got[n] is None:
            continue
        x = np.asarray(got[n], dtype=np.float64)
        assert x.shape == w.shape, (n, x.shape, w.shape)
        m, there = mag[n], ~np.isnan(w)
        kind = name if n in ("y", "dq", "dk", "dv") else "f32"
        err = count * U * m
        if n == "dg":
            err = err + 256.0 * U * chunk_sums(a, mag, spans)
        if kind != "f32":
            err = err + HALF_STEP[kind] * m * (1.0 + 2.0 * count * U)
            if kind == "f16":
                # factors scaled to float16's range keep 2^-39 of the largest
                err = err + 2.0 ** -30 * np.nanmax(np.where(there, m, 0.0), initial=0.0)
        tol = HALF_STEP[kind] * (np.abs(w) + err) + err + SMALLEST[kind]
        near = np.abs(x - w) <= tol
        if kind == "f16":
            # float16 ends at 65504 = 2^16 - 2^5: from half a step (2^4) beyond, 65520, a result is an infinity
            near |= np.isinf(x) & (x * w > 0) & (np.abs(w) + tol >= 65520.0)
        bad = there & ~near
        if bad.any():
            at = tuple(int(v[0]) for v in np.nonzero(bad))
            raise AssertionError(f"{what} {n}: {int(bad.sum())} of {int(there.sum())} off, first at {at}: {x[at]} for "
                                 f"{w[at]}, tolerance {tol[at]:.3g}")
        if kind == "f32" and n not in ("dD", "dg") and there.any():
            off, norm = np.linalg.norm((x - w)[there]), np.linalg.norm(w[there])
            assert off <= 64 * U * norm + 64 * U * np.linalg.norm(m[there]) / np.sqrt(64.0), (what, n, off / norm)


def chunk_sums(a, mag, spans):
    """What meets in dg's running sums: W over a chunk's pairs and with the states beside it, by its rows
    (q . dq) and columns (beta dbeta), per head; broadcast over the 64 steps around each."""
    H, G = a["v"].shape[1], a["q"].shape[1]
    of = np.arange(H) // (H // G)
    rows = (np.abs(a["q"]) * np.nan_to_num(mag["dq"])).sum(2)[:, of]
    beta = 1.0 if a["beta"] is None else np.abs(a["beta"])
    columns = beta * np.nan_to_num(mag["dbeta"])
    each = rows + columns
    out = np.zeros_like(each)
    for t in range(each.shape[2]):
        out[:, :, t] = each[:, :, max(0, t - 63):t + 64].sum(2)
    return out + np.nan_to_num(mag["dg"])


def call_args(a, name, order, dev="cuda:0"):
    """(positional arguments, keywords) of ssm.linear_attention"""
    import torch
    f32 = lambda v: None if v is None else torch.from_numpy(np.asarray(v)).float().to(dev)  # noqa: E731
    args = [on_device(a[n], name, order, dev) for n in ("q", "k", "v")] + [f32(a["g"])]
    return args, dict(beta=f32(a["beta"]), D=f32(a["D"]), scale=a["scale"], x0=f32(a["x0"]))
