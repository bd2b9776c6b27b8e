"""Bounds on what float32 rounding does to the selective scan and its gradients.

The rounding errors are carried through the recurrence itself: an error made at a
step decays with the states behind it.  All counts are half steps of float32
(2^-24 relative): an addition, product or multiply-add is one, the hardware's
exponential, logarithm and reciprocal are two each (one unit).

    dt      the sum v = delta + bias is off by |v| (the slope of softplus is at most
            softplus itself), its exponential by |v| for the product with log2(e)
            and 4 more, the logarithm with its correction and the products by 8:
            2 |v| + 14; without softplus 2
    decay   exp2(dt A2): A2 by 2, the product by 1, dt by its own, all times the
            exponent |dt A|, and 2; where chunks are folded, dt is a sum, of ADDS terms at most
    x_t     the decay's error times what decays, dt + 2 on dt u B, 1 on the state
    C . x   18: a lane's states one by one, three levels of lanes
    gate    z sigmoid(z): |z| + 12, p = dy silu(z) the same
    g_t, carry   as x_t, from the end

Magnitudes add up absolute values; second-order terms are below the counts' slack."""
import numpy as np

import oracle.selective_oracle as S

U = 2.0 ** -24
ADDS = 64   # additions in a chunk's sum of dt: one per tile, then 32 threads' parts


def _dense(a, dy, dlast, L, blocks):
    """One call on n rows of L steps each; arrays [n, ...] as in the oracle."""
    u, delta, A, B, C = a["u"], a["delta"], a["A"], a["B"], a["C"]
    n, H, _ = u.shape
    N, G = A.shape[1], B.shape[1]
    rep = H // G
    bias = np.zeros(H) if a["bias"] is None else a["bias"]
    D = np.zeros(H) if a["D"] is None else np.abs(a["D"])
    v = delta + bias[:, None]
    dt = S.softplus(v) if a["soft"] else v
    slope = S.sigmoid(v) if a["soft"] else np.ones_like(v)
    r_dt = 2.0 * np.abs(v) + 14.0 if a["soft"] else np.full_like(v, 2.0)
    adt, au = np.abs(dt), np.abs(u)
    wide = lambda w, t: np.repeat(np.abs(w[:, :, :, t]), rep, 1)  # noqa: E731
    x = np.zeros((n, H, N)) if a["x0"] is None else np.abs(a["x0"])
    err = np.zeros((n, H, N))
    xs, es, decs, cs = [x], [err], [], []
    pre, pre_err = np.zeros((n, H, L)), np.zeros((n, H, L))
    for t in range(L):
        d, E = dt[:, :, t, None], np.abs(dt[:, :, t, None] * A)
        dec, c = np.exp(d * A), E * (3.0 + r_dt[:, :, t, None] + ADDS) + 2.0
        dxB = (adt[:, :, t] * au[:, :, t])[..., None] * wide(B, t)
        new = dec * x + dxB
        err = dec * err + U * (c * dec * x + (r_dt[:, :, t, None] + 2.0) * dxB + new)
        x = new
        pre[:, :, t] = (wide(C, t) * x).sum(2) + D * au[:, :, t]
        pre_err[:, :, t] = (wide(C, t) * err).sum(2) + 18.0 * U * pre[:, :, t]
        xs.append(x), es.append(err), decs.append(dec), cs.append(c)
    if a["z"] is None:
        out = dict(y=pre_err, x=err)
        gate, r_p = 1.0, 0.0
    else:
        az, s = np.abs(a["z"]), S.sigmoid(a["z"])
        gate, r_p = az * s, az + 12.0
        out = dict(y=gate * (pre_err + U * r_p * pre), x=err)
    if dy is None:
        return out
    ady = np.abs(dy)
    p = ady * gate
    r_p = np.broadcast_to(r_p, p.shape)
    if a["z"] is not None:
        off = s * (1.0 + az) * (az + 12.0)   # of the slope of silu
        out["dz"] = ady * (1.1 * pre_err + U * pre * (off + 3.3))
    du, ddt, dd_mag = np.zeros((n, H, L)), np.zeros((n, H, L)), np.zeros((n, H, L))
    dB, dC = np.zeros((n, G, N, L)), np.zeros((n, G, N, L))
    dA, dA_mag = np.zeros((H, N)), np.zeros((H, N))
    carry = np.zeros((n, H, N)) if dlast is None else np.abs(dlast)
    cerr = np.zeros((n, H, N))
    over = 16.0 + blocks   # additions over channels: lanes, waves, workgroups
    for t in range(L - 1, -1, -1):
        pt, rp, rd = p[:, :, t, None], r_p[:, :, t, None], r_dt[:, :, t, None]
        Bt, Ct, d, dx = wide(B, t), wide(C, t), adt[:, :, t, None], (adt * au)[:, :, t, None]
        g = carry + pt * Ct
        gerr = cerr + U * (rp * pt * Ct + g)
        sums = lambda w: w.reshape(n, G, rep, N).sum(2)  # noqa: E731
        dB[..., t] = sums(gerr * dx + U * (rd + 2.0 + over) * g * dx)
        dC[..., t] = sums(pt * es[t + 1] + U * (rp + 1.0 + over) * pt * xs[t + 1])
        gB, gB_err = (g * Bt).sum(2), (gerr * Bt).sum(2)
        gB_err = gB_err + 18.0 * U * gB
        cerr = decs[t] * (gerr + U * (cs[t] + 1.0) * g)
        carry = decs[t] * g
        back = carry * xs[t]
        berr = cerr * xs[t] + carry * es[t] + U * back
        dA += (berr * d + U * (rd + 1.0) * back * d).sum(0)
        dA_mag += (back * d).sum(0)
        aA = np.abs(A)
        bA, bA_err = (back * aA).sum(2), (berr * aA).sum(2)
        bA_err = bA_err + 20.0 * U * bA
        pd = p[:, :, t]
        du[:, :, t] = (D * pd * r_p[:, :, t] * U + adt[:, :, t] * (gB_err + U * (r_dt[:, :, t] + 2.0) * gB)
                       + 2.0 * U * (D * pd + adt[:, :, t] * gB))
        mag = au[:, :, t] * gB + bA
        r_s = 2.0 * np.abs(v[:, :, t]) + 12.0 if a["soft"] else 0.0
        ddt[:, :, t] = slope[:, :, t] * (au[:, :, t] * gB_err + bA_err + U * (4.0 + r_s) * mag)
        dd_mag[:, :, t] = slope[:, :, t] * mag
    adds = L / 32.0 + 40.0   # of a thread that moves steps, then over threads; rows are added in float64
    out.update(du=du, ddelta=ddt, dB=dB, dC=dC, dA=dA + L * U * dA_mag, dx0=cerr,
               dD=(p * au * (r_p + 1.0 + adds)).sum((0, 2)) * U,
               ddelta_bias=ddt.sum((0, 2)) + adds * U * dd_mag.sum((0, 2)))
    return out


def scan_bounds(a, spans, dy=None, dlast=None):
    """dict of error bounds for y and the final states x (and, with dy, every
    gradient), in the oracle's shapes; steps outside every span get 0."""
    Bsz, H, L = a["u"].shape
    per_group = H // a["B"].shape[1]
    blocks = (per_group + 63) // 64
    if spans == S.dense_spans(Bsz, L):
        return _dense(a, dy, dlast, L, blocks)
    out = None
    for i, (row, beg, end) in enumerate(spans):
        cut = {k: w[row:row + 1, ..., beg:end] if k in ("u", "delta", "B", "C") or (k == "z" and w is not None) else w
               for k, w in a.items()}
        cut["x0"] = None if a["x0"] is None else a["x0"][i:i + 1]
        one = _dense(cut, None if dy is None else dy[row:row + 1, :, beg:end],
                     None if dlast is None else dlast[i:i + 1], end - beg, blocks)
        if out is None:
            whole = dict(y=a["u"].shape, dz=a["u"].shape, du=a["u"].shape, ddelta=a["u"].shape, dB=a["B"].shape,
                         dC=a["C"].shape, x=(len(spans), H, a["A"].shape[1]), dx0=(len(spans), H, a["A"].shape[1]))
            out = {k: np.zeros(whole.get(k, w.shape)) for k, w in one.items()}
        for k, w in one.items():
            if k in ("x", "dx0"):
                out[k][i] = w[0]
            elif k in ("dA", "dD", "ddelta_bias"):
                out[k] += w
            else:
                out[k][row, ..., beg:end] = w[0]
    return out


def within(got, want, err, name, what):
    """|got - want| <= err, and half a step of the output's type."""
    from tests import selective_cases as K
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    there = ~np.isnan(want)
    tol = K.HALF_STEP[name] * (np.abs(want) + err) + err + K.SMALLEST[name]
    bad = there & ~(np.abs(got - want) <= tol)
    if bad.any():
        at = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(there.sum())} off, first at {at}: "
                             f"{got[at]} for {want[at]}, tolerance {tol[at]:.3g}")
