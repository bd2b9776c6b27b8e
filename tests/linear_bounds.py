"""Bounds on the norm of linear attention's errors, from what independent roundings add up
to (their root, not their sum): tighter than the elementwise bounds of tests/linear_cases.py,
so that a systematic rounding, a lost part of an operand or a scale that is off by a little
does not pass.  Everything is per head: the oracle runs with each head's own copy of its
group's queries and keys.

A rounding to the type is off by at most half a step, HALF_STEP relative, anywhere within it
alike: a third of its square on average.  In float32 an element's sums have the
roundings of three exponents (4 D, D the most that |g| adds up to over 64 steps), 16 of
exponentials and products and 2 sqrt(64) of additions: COUNT = 32 + 4 D half steps, U each.

dg_r   is a running sum over its chunk of R_t - C_s (R_t = q_t . dq_t, C_s = beta_s dbeta_s, of
       the head) and of <x, X>.  R and C are sums of signed terms: what rounding does to them is
       relative to the root of their terms' squares, which the sums themselves have on average.
dD     sums of dy v, COUNT relative to the root of their squares.
y, dv, dq, dk   one rounding of the result.  The weights of pairs and the states are operands in two
       parts of the type: the square of its half step, relative to the terms M_ts v_s, x_np q_n and
       u_ts beta_s dM_ts k_s, beside COUNT half steps of float32."""
import numpy as np

import oracle.linear_oracle as O
from tests.linear_cases import HALF_STEP, U


def chunk(name):
    return 32 if name == "f32" else 64


def count(a):
    L = a["g"].shape[2]
    g = np.where(np.isinf(a["g"]), 0.0, np.abs(a["g"]))
    total = np.cumsum(np.concatenate([np.zeros((*g.shape[:2], 1)), g], 2), 2)
    D = (total[:, :, 64:] - total[:, :, :-64]).max() if L >= 64 else total[:, :, -1].max()
    return 32.0 + 4.0 * D


def per_head(a):
    H, G = a["v"].shape[1], a["q"].shape[1]
    of = np.arange(H) // (H // G)
    return {**a, "q": a["q"][:, of], "k": a["k"][:, of]}


def over_chunks(each, name, spans):
    """The root of what `each` [Bsz, H, L] adds up to over the chunk around every step."""
    out, Q = np.zeros_like(each), chunk(name)
    for row, beg, end in spans:
        for t in range(beg, end, Q):
            e = min(t + Q, end)
            out[row, :, t:e] = np.sqrt(each[row, :, t:e].sum(1))[:, None]
    return out


def decay_sums(a, name, spans):
    """dict of norms: what dg and dD may be off by."""
    b = per_head(a)
    g = O.attention_grad(b["q"], b["k"], b["v"], b["g"], b["beta"], b["D"], b["scale"], b["x0"], b["dy"], b["dx"], spans)
    rows = (b["q"] * np.nan_to_num(g["dq"])).sum(2)
    columns = (1.0 if b["beta"] is None else b["beta"]) * np.nan_to_num(g["dbeta"])
    c = count(a) * U
    terms = np.zeros(a["v"].shape[1])
    for row, beg, end in spans:
        terms += ((a["dy"] * a["v"])[row, :, :, beg:end] ** 2).sum((1, 2))
    return dict(dg=c * (np.linalg.norm(over_chunks(rows ** 2 + columns ** 2, name, spans)) + np.linalg.norm(np.nan_to_num(g["dg"]))),
                dD=c * (np.linalg.norm(np.sqrt(terms)) + np.linalg.norm(g["dD"])))


def results(a, name, spans):
    """dict of norms: what y, dv, dq and dk of a 16-bit type may be off by."""
    b, Q, H = per_head(a), chunk(name), a["v"].shape[1]
    G = a["q"].shape[1]
    of = np.arange(H) // (H // G)
    y, _, states = O.attention(b["q"], b["k"], b["v"], b["g"], b["beta"], b["D"], b["scale"], b["x0"], spans)
    grads = O.attention_grad(a["q"], a["k"], a["v"], a["g"], a["beta"], a["D"], a["scale"], a["x0"], a["dy"], a["dx"], spans)
    sq = dict(y=0.0, dv=0.0, dq=0.0, dk=0.0)
    for s, (row, beg, end) in enumerate(spans):
        X = np.zeros((H, a["q"].shape[2], a["v"].shape[2])) if a["dx"] is None else a["dx"][s].copy()
        for t0 in reversed(range(beg, end, Q)):
            t1 = min(t0 + Q, end)
            q, k, v, dy = (b[n][row, :, :, t0:t1] for n in ("q", "k", "v", "dy"))
            g, beta = b["g"][row, :, t0:t1], np.ones((H, t1 - t0)) if b["beta"] is None else b["beta"][row, :, t0:t1]
            run = np.cumsum(np.where(np.isinf(g), -1e4, g), 1)
            E = np.tril(np.exp(np.minimum(run[:, :, None] - run[:, None, :], 700.0))) * a["scale"] * beta[:, None, :]
            M = np.einsum("hnt,hns->hts", q, k) * E
            dM = np.einsum("hpt,hps->hts", dy, v) * E
            before = np.zeros_like(X) if t0 == beg and a["x0"] is None else a["x0"][s] if t0 == beg else states[s, t0 - 1]
            from_, to = np.exp(run) * a["scale"], np.exp(run[:, -1:] - run) * beta
            sq["y"] += np.einsum("hts,hps->", M ** 2, v ** 2) + np.einsum("hnp,hnt,ht->", before ** 2, q ** 2, from_ ** 2)
            sq["dv"] += np.einsum("hts,hpt->", M ** 2, dy ** 2) + np.einsum("hnp,hns,hs->", X ** 2, k ** 2, to ** 2)
            sq["dq"] += np.einsum("hts,hns->", dM ** 2, k ** 2)
            sq["dk"] += np.einsum("hts,hnt->", dM ** 2, q ** 2)
            for t in range(t1 - 1, t0 - 1, -1):      # the gradient of the state in front of the chunk
                X = np.exp(b["g"][row, :, t])[:, None, None] * (
                    X + a["scale"] * b["q"][row, :, :, t][:, :, None] * b["dy"][row, :, :, t][:, None, :])
    whole = dict(y=y, dv=grads["dv"], dq=grads["dq"], dk=grads["dk"])
    half, fine = HALF_STEP[name] / np.sqrt(3.0), HALF_STEP[name] ** 2 + count(a) * U
    return {n: half * np.sqrt(np.nansum(whole[n] ** 2)) * (1.0 + 2.0 ** -5) + fine * np.sqrt(sq[n]) for n in sq}


def off(got, want):
    there = ~np.isnan(want)
    return float(np.linalg.norm((got - want)[there]))
