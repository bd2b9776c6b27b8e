"""Float64 definitions of the selective operators (numpy, one step at a time),
and their gradients by the chain rule.

Arrays are [Bsz, H, L] (B and C [Bsz, G, N, L]); `spans` lists the sequences as
(row, begin, end) along the rows' steps.  Steps outside every span keep NaN in
the outputs, which the tests read as "not written".

Every function also runs on the absolute values of its inputs with `mag=True`:
each product and sum then adds up magnitudes, which bounds what float32
rounding can do to the same sum (used for tolerances only)."""
import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def silu(v):
    return v * sigmoid(v)


def silu_slope(v):
    p = sigmoid(v)
    return p * (1.0 + v * (1.0 - p))


def softplus(v):
    return np.logaddexp(v, 0.0)


def dense_spans(Bsz, L, lengths=None):
    return [(b, 0, L if lengths is None else int(lengths[b])) for b in range(Bsz)]


def packed_spans(offsets):
    return [(0, int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


# ------------------------------------------------------------- convolution ----

def conv(u, w, bias, act, state, spans):
    """(y, final states): pre_t = bias + sum_k w[k] u_{t-W+1+k}, y = silu(pre) or pre."""
    H, W = w.shape
    y = np.full(u.shape, np.nan)
    last = np.zeros((len(spans), H, W - 1))
    for s, (row, beg, end) in enumerate(spans):
        past = np.zeros((H, W - 1)) if state is None else state[s]
        line = np.concatenate([past, u[row, :, beg:end]], 1)
        for t in range(end - beg):
            pre = (line[:, t:t + W] * w).sum(1) + (0.0 if bias is None else bias)
            y[row, :, beg + t] = silu(pre) if act else pre
        last[s] = line[:, line.shape[1] - (W - 1):]
    return y, last


def conv_grad(u, w, bias, act, state, dy, dlast, spans, mag=False):
    """dict(du, dweight, dbias, dstate): gradients for dy of y and dlast of the final states."""
    H, W = w.shape
    m = np.abs if mag else (lambda v: v)
    du, dw, db = np.full(u.shape, np.nan), np.zeros_like(w), np.zeros(H)
    dstate = np.zeros((len(spans), H, W - 1))
    for s, (row, beg, end) in enumerate(spans):
        past = np.zeros((H, W - 1)) if state is None else state[s]
        line = np.concatenate([past, u[row, :, beg:end]], 1)
        dline = np.zeros_like(line)
        if dlast is not None:
            dline[:, line.shape[1] - (W - 1):] += m(dlast[s])
        for t in range(end - beg):
            pre = (line[:, t:t + W] * w).sum(1) + (0.0 if bias is None else bias)
            d = m(dy[row, :, beg + t])
            if act:  # |slope| <= 1.1, and its own error counts relative to 1
                d = d * (1.1 if mag else silu_slope(pre))
            dline[:, t:t + W] += d[:, None] * m(w)
            dw += d[:, None] * m(line[:, t:t + W])
            db += d
        dstate[s] = dline[:, :W - 1]
        du[row, :, beg:end] = dline[:, W - 1:]
    return dict(du=du, dweight=dw, dbias=db, dstate=dstate)


# -------------------------------------------------------------------- scan ----

def _dt(delta, bias, soft):
    v = delta + (0.0 if bias is None else bias[:, None])
    return softplus(v) if soft else v


def scan(u, delta, A, B, C, D, z, bias, soft, x0, spans, mag=False):
    """(y, final states, states after every step [Bsz, L, H, N])."""
    Bsz, H, L = u.shape
    N, G = A.shape[1], B.shape[1]
    m = np.abs if mag else (lambda v: v)
    rep = H // G
    dt = _dt(delta, bias, soft)
    y = np.full(u.shape, np.nan)
    xs = np.full((Bsz, L, H, N), np.nan)
    last = np.zeros((len(spans), H, N))
    for s, (row, beg, end) in enumerate(spans):
        x = np.zeros((H, N)) if x0 is None else m(x0[s]).copy()
        for t in range(beg, end):
            Bt, Ct = (np.repeat(m(v[row, :, :, t]), rep, 0) for v in (B, C))
            d = dt[row, :, t]
            x = np.exp(d[:, None] * A) * x + m(d * u[row, :, t])[:, None] * Bt
            xs[row, t] = x
            o = (x * Ct).sum(1)
            if D is not None:
                o = o + m(D * u[row, :, t])
            if z is not None:
                o = o * m(silu(z[row, :, t]))
            y[row, :, t] = o
        last[s] = x
    return y, last, xs


def scan_grad(u, delta, A, B, C, D, z, bias, soft, x0, dy, dlast, spans, mag=False):
    """dict of every gradient for dy of y and dlast of the final states."""
    Bsz, H, L = u.shape
    N, G = A.shape[1], B.shape[1]
    m = np.abs if mag else (lambda v: v)
    rep = H // G
    dt = _dt(delta, bias, soft)
    v = delta + (0.0 if bias is None else bias[:, None])
    slope = sigmoid(v) if soft else np.ones_like(v)
    _, _, xs = scan(u, delta, A, B, C, D, None, bias, soft, x0, spans, mag)
    du, ddt, dz = (np.full(u.shape, np.nan) for _ in range(3))
    dB, dC = np.full(B.shape, np.nan), np.full(C.shape, np.nan)
    dA, dD, dx0 = np.zeros_like(A), np.zeros(H), np.zeros((len(spans), H, N))
    for s, (row, beg, end) in enumerate(spans):
        start = np.zeros((H, N)) if x0 is None else m(x0[s])
        carry = np.zeros((H, N)) if dlast is None else m(dlast[s]).copy()
        for t in range(end - 1, beg - 1, -1):
            Bt, Ct = (np.repeat(m(w[row, :, :, t]), rep, 0) for w in (B, C))
            x, before = xs[row, t], start if t == beg else xs[row, t - 1]
            ut, d = m(u[row, :, t]), dt[row, :, t]
            p = m(dy[row, :, t])
            if z is not None:
                pre = (x * Ct).sum(1) + (0.0 if D is None else m(D) * ut)
                dz[row, :, t] = p * pre * (1.1 if mag else silu_slope(z[row, :, t]))
                p = p * m(silu(z[row, :, t]))
            g = carry + p[:, None] * Ct
            dC[row, :, :, t] = (p[:, None] * x).reshape(G, rep, N).sum(1)
            dB[row, :, :, t] = (g * m(d * u[row, :, t])[:, None]).reshape(G, rep, N).sum(1)
            gB = (g * Bt).sum(1)
            carry = np.exp(d[:, None] * A) * g
            back = carry * before
            du[row, :, t] = m(d) * gB + (0.0 if D is None else m(D) * p)
            ddt[row, :, t] = ((back * m(A)).sum(1) + ut * gB) * slope[row, :, t]
            dA += back * m(d)[:, None]
            dD += p * ut
        dx0[s] = carry
    out = dict(du=du, ddelta=ddt, dA=dA, dB=dB, dC=dC, dD=dD, ddelta_bias=np.nansum(ddt, (0, 2)), dx0=dx0)
    if z is not None:
        out["dz"] = dz
    return out
