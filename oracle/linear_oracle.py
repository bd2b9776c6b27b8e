"""Float64 definitions of linear attention with a decay for each head and of layer
norm (numpy, one step at a time), and their gradients by the chain rule.

Attention: q, k [Bsz, G, N, L], v [Bsz, H, P, L], g, beta [Bsz, H, L] (beta or None),
D [H] or None; `spans` lists the sequences as (row, begin, end) along the rows'
steps.  Steps outside every span keep NaN in the outputs, which the tests read as
"not written".

With `mag=True` the attention functions add up magnitudes (decays as they are): a
bound on what rounding can do to the same sums, used for tolerances only."""
import numpy as np


def _parts(q, k, v, row, t, scale, beta, m):
    H, G = v.shape[1], q.shape[1]
    of = np.arange(H) // (H // G)
    qt, kt = m(q[row, of, :, t]) * abs(scale) if m is np.abs else q[row, of, :, t] * scale, m(k[row, of, :, t])
    return qt, kt, m(v[row, :, :, t]), np.ones(H) if beta is None else m(beta[row, :, t])


def attention(q, k, v, g, beta, D, scale, x0, spans, mag=False):
    """(y, final states [S, H, N, P], states after every step as a dict (sequence, t))."""
    H, P, N = v.shape[1], v.shape[2], q.shape[2]
    m = np.abs if mag else (lambda a: a)
    y = np.full(v.shape, np.nan)
    last, states = np.zeros((len(spans), H, N, P)), {}
    for s, (row, beg, end) in enumerate(spans):
        x = np.zeros((H, N, P)) if x0 is None else m(x0[s]).copy()
        for t in range(beg, end):
            qt, kt, vt, b = _parts(q, k, v, row, t, scale, beta, m)
            x = np.exp(g[row, :, t])[:, None, None] * x + (b[:, None] * kt)[:, :, None] * vt[:, None, :]
            states[s, t] = x
            y[row, :, :, t] = np.einsum("hn,hnp->hp", qt, x) + (0.0 if D is None else m(D)[:, None] * vt)
        last[s] = x
    return y, last, states


def attention_grad(q, k, v, g, beta, D, scale, x0, dy, dlast, spans, mag=False):
    """dict of every gradient for dy of y and dlast of the final states."""
    H, P, N, G = v.shape[1], v.shape[2], q.shape[2], q.shape[1]
    m = np.abs if mag else (lambda a: a)
    of = np.arange(H) // (H // G)
    _, _, states = attention(q, k, v, g, beta, D, scale, x0, spans, mag)
    dq, dk, dv = (np.full(a.shape, np.nan) for a in (q, k, v))
    dg, dbeta = np.full(g.shape, np.nan), np.full(g.shape, np.nan)
    dD, dx0 = np.zeros(H), np.zeros((len(spans), H, N, P))
    for s, (row, beg, end) in enumerate(spans):
        dq[row, :, :, beg:end] = dk[row, :, :, beg:end] = 0.0
        start = np.zeros((H, N, P)) if x0 is None else m(x0[s])
        X = np.zeros((H, N, P)) if dlast is None else m(dlast[s]).copy()
        for t in range(end - 1, beg - 1, -1):
            qt, kt, vt, b = _parts(q, k, v, row, t, scale, beta, m)
            d = m(dy[row, :, :, t])
            x, before = states[s, t], start if t == beg else states[s, t - 1]
            X = X + qt[:, :, None] * d[:, None, :]
            e = np.exp(g[row, :, t])
            np.add.at(dq[row, :, :, t], of, abs(scale) * np.einsum("hnp,hp->hn", x, d) if mag
                      else scale * np.einsum("hnp,hp->hn", x, d))
            Xv, Xk = np.einsum("hnp,hp->hn", X, vt), np.einsum("hnp,hn->hp", X, kt)
            np.add.at(dk[row, :, :, t], of, b[:, None] * Xv)
            dv[row, :, :, t] = b[:, None] * Xk + (0.0 if D is None else m(D)[:, None] * d)
            dbeta[row, :, t] = (kt * Xv).sum(1)
            dg[row, :, t] = e * (X * before).sum((1, 2))
            dD += (d * vt).sum(1)
            X = e[:, None, None] * X
        dx0[s] = X
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, dD=dD, dx0=dx0)


# -------------------------------------------------------------- layer norm ----

def _sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def norm(u, weight, bias, z, gate, rms, groups, eps):
    """(y, the normed numbers, 1 / root) for u, z [Bsz, H, L]."""
    Bsz, H, L = u.shape
    a = u * z * _sigmoid(z) if z is not None and gate == "before" else u
    a = a.reshape(Bsz, groups, H // groups, L)
    if not rms:
        a = a - a.mean(2, keepdims=True)
    r = 1.0 / np.sqrt((a * a).mean(2, keepdims=True) + eps)
    n = (a * r).reshape(Bsz, H, L)
    y = n * (1.0 if weight is None else weight[:, None]) + (0.0 if bias is None else bias[:, None])
    if z is not None and gate == "after":
        y = y * z * _sigmoid(z)
    return y, n, r


def norm_grad(u, dy, weight, bias, z, gate, rms, groups, eps):
    """dict of every gradient for dy of y."""
    Bsz, H, L = u.shape
    _, n, r = norm(u, weight, bias, z, gate, rms, groups, eps)
    w = np.ones(H) if weight is None else weight
    out, d = {}, dy
    if z is not None:
        p = _sigmoid(z)
        slope = p * (1.0 + z * (1.0 - p))
        if gate == "after":
            out["dz"] = dy * (n * w[:, None] + (0.0 if bias is None else bias[:, None])) * slope
            d = dy * z * p
    out["dweight"], out["dbias"] = (d * n).sum((0, 2)), d.sum((0, 2))
    shape = (Bsz, groups, H // groups, L)
    dn, m = (d * w[:, None]).reshape(shape), n.reshape(shape)
    da = dn - m * (dn * m).mean(2, keepdims=True)
    if not rms:
        da = da - dn.mean(2, keepdims=True)
    da = (da * r).reshape(u.shape)
    if z is not None and gate == "before":
        out["dz"] = da * u * slope
        da = da * z * p
    out["du"] = da
    return out
