"""Linear attention with a decay for each head, and layer norm, as cases that can be timed and checked.

Per head h with keys of N and values of P numbers, q and k shared by the heads of a group:

    x_t = exp(g_t) x_{t-1} + beta_t k_t v_t^T          (a state of N x P)
    y_t = scale x_t^T q_t + D v_t

for whole prompts (dense, or packed one behind the other), for training (with
every gradient) and for single tokens on states that live in a pool of slots;
and, over the channels of a group at every step,

    n = (a - mean a) / sqrt(var a + eps)   or   n = a / sqrt(mean a^2 + eps)
    y = n weight + bias

with the gate silu(z) on the input (a = u silu(z)) or on the output, forward and
backward.

`run` computes them in elementary torch operations, in 32 bits, rounded once
at the end; with `own` set it calls the library's entry points.  Activations
are [batch, ..., steps] in either order of storage ("rows": steps contiguous,
"tokens": channels contiguous).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CHUNK = 64      # steps that the plain form takes at a time
EPS = 1e-5


# ---------------------------------------------------------------- cases ----

def _attention(name, op, dtype, batch, heads, keys, values, steps=1, groups=1, order="tokens", packed="",
               decay="token", beta=True, skip=True, carry=False, pool=0):
    c = dict(op=op, dtype=dtype, batch=batch, heads=heads, keys=keys, values=values, steps=steps, groups=groups,
             order=order, packed=packed, decay=decay, beta=beta, skip=skip, carry=carry, pool=pool)
    if name:
        c["name"] = name
    return c


def _norm(name, op, dtype, batch, channels, steps=1, groups=1, order="tokens", rms=True, gate="", bias=False):
    c = dict(op=op, dtype=dtype, batch=batch, channels=channels, steps=steps, groups=groups, order=order, rms=rms,
             gate=gate, bias=bias)
    if name:
        c["name"] = name
    return c


def listed():
    prompts = "1,0,517,1300,64,3,2215,996"     # a serving batch: an empty and a one-token prompt, odd lengths
    return [
        # one long prompt, its heads' keys and queries shared
        _attention("attention long prompt", "attend", "bf16", 1, 32, 128, 64, 16384),
        # continued prompts of a serving batch packed one behind the other, on their states
        _attention("attention packed prompts", "attend", "f16", 1, 24, 64, 64, 5096, packed=prompts, carry=True),
        # a training step: forward with what the backward pass needs, then every gradient
        _attention("attention training", "attend_train", "bf16", 4, 64, 128, 64, 2048),
        # the same in single precision at the filter path's s4-h256-l1k sizes and storage order, states carried over
        _attention("attention training rows", "attend_train", "f32", 8, 4, 64, 64, 1024, groups=2, order="rows",
                   carry=True),
        # heads with keys of their own and fixed decays, an odd length
        _attention("attention training heads", "attend_train", "bf16", 2, 16, 128, 128, 1500, groups=16, decay="head",
                   beta=False, skip=False),
        # one sequence's next token: latency
        _attention("attention one token", "attend_step", "bf16", 1, 32, 128, 64, pool=1),
        # a large decode batch on a pool of slots
        _attention("attention decode batch", "attend_step", "bf16", 250, 64, 128, 64, pool=256),
        # the gated norm behind a long prompt's scan
        _norm("norm long prompt", "norm", "bf16", 1, 2048, 16384, gate="before"),
        # a training step of it
        _norm("norm training", "norm_train", "bf16", 4, 4096, 2048, gate="before"),
        # with mean and bias in single precision at the filter path's s4-h512-l3k sizes and storage order
        _norm("norm training rows", "norm_train", "f32", 16, 512, 3000, order="rows", rms=False, bias=True),
        # one sequence's next token: latency
        _norm("norm one token", "norm", "bf16", 1, 2048, gate="before"),
        # a large decode batch, each head normed by itself and gated behind
        _norm("norm decode batch", "norm", "f16", 250, 8192, groups=128, rms=False, gate="after", bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    if c["op"].startswith("norm"):
        return c["batch"] * c["channels"] * c["steps"] * (2 if c["dtype"] == "f32" else 1)
    # the plain form's products and its tables of a chunk's decays
    N, P = c["keys"], c["values"]
    return (c["batch"] * c["heads"] * (c["steps"] + (CHUNK * c["packed"].count(",") if c["packed"] else 0))
            * (N * P + CHUNK * (N + P) + 32 * CHUNK) * (2 if c["dtype"] == "f32" else 1))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend_train", "attend_train", "attend_step", "norm", "norm_train"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    while True:
        order = rng.choice(["tokens", "tokens", "rows"])
        if op.startswith("norm"):
            groups = rng.choice([1, 1, 2, 8])
            channels = groups * _log_int(rng, max(16, 64 // groups), 8192 // groups)
            c = _norm("", op, dtype, _log_int(rng, 1, 256), channels, _log_int(rng, 1, 16384), groups, order,
                      rng.random() < 0.6, rng.choice(["", "before", "after"]), rng.random() < 0.5)
        else:
            groups = rng.choice([1, 1, 2, 4])
            heads = groups * _log_int(rng, 1, 96 // groups)
            if rng.random() < 0.25:
                groups = heads
            keys = rng.choice([16, 32, 64, 64, 128, 128, 256, rng.randrange(17, 200)])
            values = rng.choice([32, 64, 64, 64, 128, 256, rng.randrange(17, 200)])
            more = dict(groups=groups, decay=rng.choice(["token", "token", "head"]), beta=rng.random() < 0.7,
                        skip=rng.random() < 0.6)
            if op == "attend_step":
                batch = _log_int(rng, 1, 256)
                c = _attention("", op, dtype, batch, heads, keys, values, pool=batch + rng.randrange(1, 17), **more)
            else:
                steps, batch, packed = _log_int(rng, 50, 16384), _log_int(rng, 1, 16), ""
                if op == "attend" and rng.random() < 0.4:
                    count, batch, order = rng.randrange(2, 12), 1, "tokens"
                    cuts = sorted(rng.randrange(0, steps + 1) for _ in range(count - 1))
                    packed = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [steps]))
                c = _attention("", op, dtype, batch, heads, keys, values, steps, order=order, packed=packed,
                               carry=rng.random() < 0.5, **more)
        if _cost(c) <= most:
            return c


# --------------------------------------------------------------- inputs ----

def _lengths(c):
    return [int(v) for v in c["packed"].split(",")] if c.get("packed") else []


def _plan(c, offsets, lens):
    """The chunks of a call, as a plain program lays them out: for each the places of its steps along
    the row (`at`, where `live`), its sequence and that one's first chunk; for each step its place among
    the chunks' steps; for each sequence its last chunk."""
    at, live, seq, first, last, back = [], [], [], [], [], []
    for s, (begin, n) in enumerate(zip(offsets, lens)):
        start = len(at)
        for k in range(max(1, -(-n // CHUNK))):
            places = list(range(k * CHUNK, (k + 1) * CHUNK))
            at.append([begin + p if p < n else 0 for p in places])
            live.append([p < n for p in places])
            back += [len(seq) * CHUNK + i for i, p in enumerate(places) if p < n]
            seq.append(s)
            first.append(start)
        last.append(len(at) - 1)
    t = lambda v: torch.tensor(v, device=DEV)  # noqa: E731
    return dict(at=t(at), live=t(live), seq=t(seq), first=t(first), last=t(last), back=t(back))


def prepare(case, seed):
    c, t = case, DTYPES[case["dtype"]]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=DEV) * scale

    def act(Bsz, *rest):
        # [batch, ..., steps] of the activations' type; in "tokens" order the steps' axis is stored first
        if c["order"] == "tokens":
            return normal(Bsz, rest[-1], *rest[:-1]).to(t).movedim(1, -1)
        return normal(Bsz, *rest).to(t)

    Bsz, L, G = c["batch"], c["steps"], c["groups"]
    if c["op"].startswith("norm"):
        H = c["channels"]
        s = dict(case=c, u=act(Bsz, H, L), z=act(Bsz, H, L) if c["gate"] else None,
                 weight=1.0 + normal(H, scale=0.2), bias=normal(H, scale=0.2) if c["bias"] else None)
        if c["op"] == "norm_train":
            s["dy"] = act(Bsz, H, L)
        return s
    H, N, P = c["heads"], c["keys"], c["values"]
    s = dict(case=c, scale=1.0 / math.sqrt(N))
    if c["order"] == "tokens":
        # slices of what one projection and convolution write
        wide = normal(Bsz, L, H * P + 2 * G * N).to(t)
        s["v"] = wide[..., :H * P].unflatten(-1, (H, P)).movedim(1, -1)
        s["k"] = wide[..., H * P:H * P + G * N].unflatten(-1, (G, N)).movedim(1, -1)
        s["q"] = wide[..., H * P + G * N:].unflatten(-1, (G, N)).movedim(1, -1)
    else:
        s["v"], s["k"], s["q"] = act(Bsz, H, P, L), act(Bsz, G, N, L), act(Bsz, G, N, L)
    if c["decay"] == "token":
        # steps log-uniform in [1e-3, 1e-1] times a spread by token, rates from 1 to 16: memories of 1 to 1000 steps
        lo, hi = math.log(1e-3), math.log(1e-1)
        dt = torch.exp(lo + (hi - lo) * torch.rand(H, generator=g, device=DEV) + normal(Bsz, L, H, scale=0.7))
        rate = 1.0 + 15.0 * torch.rand(H, generator=g, device=DEV)
        s["g"] = (-dt * rate).transpose(1, 2)
        s["beta"] = (dt * 10.0).transpose(1, 2) if c["beta"] else None
    else:
        # a fixed decay for each head, 1 - 2^-5 to 1 - 2^-12
        s["g"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.rand(H, generator=g, device=DEV)))[None, :, None].expand(Bsz, H, L)
        s["beta"] = torch.rand(Bsz, L, H, generator=g, device=DEV).transpose(1, 2) if c["beta"] else None
    s["D"] = 1.0 + normal(H, scale=0.1) if c["skip"] else None
    if c["op"] == "attend_step":
        s["x"] = normal(c["pool"], H, N, P, scale=0.3)
        s["slots"] = torch.randperm(c["pool"], generator=g, device=DEV)[:Bsz].to(torch.int32)
        # one token: no axis of steps
        for k in ("q", "k", "v", "g", "beta"):
            s[k] = s[k][..., 0] if s[k] is not None else None
        return s
    lens = _lengths(c)
    S, offs = len(lens) or Bsz, [0]
    for n in lens:
        offs.append(offs[-1] + n)
    if lens:
        s["offsets"] = torch.tensor(offs, dtype=torch.int32, device=DEV)
    s["plan"] = _plan(c, offs[:-1], lens) if lens else _plan(c, [0], [L])
    if c["carry"]:
        s["x"] = normal(S, H, N, P, scale=0.3)
    if c["op"] == "attend_train":
        s["dy"] = act(Bsz, H, P, L)
        s["dx"] = normal(S, H, N, P, scale=0.3) if c["carry"] else None
    return s


# ------------------------------------------------- the library's calls ----

def _run_own(s):
    from structured_state_space_amd import ssm
    c = s["case"]
    if c["op"].startswith("norm"):
        more = dict(weight=s["weight"], bias=s["bias"], z=s["z"], gate=c["gate"] or "after", rms=c["rms"],
                    groups=c["groups"], eps=EPS)
        y = ssm.layer_norm(s["u"], **more)["y"]
        if c["op"] == "norm":
            return dict(y=y)
        grads = ssm.layer_norm_backward(s["u"], s["dy"], **more)
        return dict(y=y, **{k: v for k, v in grads.items() if v is not None})
    if c["op"] == "attend_step":
        out = ssm.linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["x"], beta=s["beta"], D=s["D"],
                                        scale=s["scale"], slots=s["slots"])
        return dict(y=out["y"], x=out["x"])
    args = (s["q"], s["k"], s["v"], s["g"])
    more = dict(beta=s["beta"], D=s["D"], scale=s["scale"], x0=s.get("x"))
    if c["op"] == "attend":
        out = ssm.linear_attention(*args, want_state=True, offsets=s.get("offsets"), **more)
        return dict(y=out["y"], x=out["x"])
    out = ssm.linear_attention(*args, want_state=True, save=True, **more)
    grads = ssm.linear_attention_backward(*args, s["dy"], dx=s["dx"], saved=out["saved"], **more)
    return dict(y=out["y"], x=out["x"], **{k: v for k, v in grads.items() if v is not None})


# ------------------------------------------------------ the plain forms ----

def _heads(v, H):
    """[batch, groups, ...] -> [batch, heads, ...]"""
    return v.repeat_interleave(H // v.shape[1], 1)


def _chunked(plan, v):
    """[batch, heads, n, steps] -> [batch, heads, chunks, steps of one, n], zero where there is no step"""
    return torch.where(plan["live"][..., None], v[..., plan["at"]].movedim(2, -1), 0.0)


def _attend(s, q, k, v, g, beta, D, x0):
    """(y, final states) in 32 bits, from inputs in 32 bits.  Sums of log decays are in 64: they pass a
    thousand in a long prompt, and their differences are what counts."""
    plan, H = s["plan"], s["case"]["heads"]
    packed, seq = "offsets" in s, plan["seq"]
    qc, kc, vc = _chunked(plan, _heads(q, H)), _chunked(plan, _heads(k, H)), _chunked(plan, v)
    gc = torch.where(plan["live"], g[..., plan["at"]].double(), 0.0)
    cum = gc.cumsum(-1)                                              # [batch, heads, chunks, steps]
    total = cum[..., -1]
    one = torch.ones((), device=DEV)
    wc = torch.where(plan["live"], one if beta is None else beta[..., plan["at"]], 0.0)
    # within a chunk
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    decay = torch.where(lower, cum.unsqueeze(-1) - cum.unsqueeze(-2), -math.inf).exp().float()
    y = (qc @ kc.transpose(-1, -2) * decay * (s["scale"] * wc).unsqueeze(-2)) @ vc
    if D is not None:
        y = y + D[:, None, None, None] * vc
    # what each chunk adds to the state, and the states before the chunks
    adds = (kc * (wc * (total.unsqueeze(-1) - cum).exp().float()).unsqueeze(-1)).transpose(-1, -2) @ vc
    ends = total.cumsum(-1)
    before = ends - total
    C = len(seq)
    follows = torch.ones(C, C, dtype=torch.bool, device=DEV).tril(-1) & (seq[:, None] == seq)
    passed = torch.where(follows, before.unsqueeze(-1) - ends.unsqueeze(-2), -math.inf).exp().float()
    x = (passed @ adds.flatten(-2)).unflatten(-1, adds.shape[-2:])
    if x0 is not None:
        begun = (before - before[..., plan["first"]]).exp().float()
        start = x0[seq].movedim(0, 1).unsqueeze(0) if packed else x0.unsqueeze(2)
        x = x + begun[..., None, None] * start
    y = y + (qc @ x) * (s["scale"] * cum.exp().float()).unsqueeze(-1)
    y = y.flatten(2, 3)[:, :, plan["back"]].transpose(-1, -2)
    last = (total.exp().float()[..., None, None] * x + adds)[:, :, plan["last"]]
    return y, last[0].movedim(1, 0) if packed else last[:, :, 0]


def _plain_attend(s):
    f = lambda k: None if s.get(k) is None else s[k].float()  # noqa: E731
    y, x = _attend(s, *(f(k) for k in ("q", "k", "v", "g", "beta", "D", "x")))
    return dict(y=y.to(s["v"].dtype), x=x.contiguous())


def _plain_attend_train(s):
    names = [n for n in ("q", "k", "v", "g", "beta", "D", "x") if s.get(n) is not None]
    with torch.enable_grad():
        leaf = {n: s[n].float().clone().requires_grad_() for n in names}
        y, x = _attend(s, *(leaf.get(n) for n in ("q", "k", "v", "g", "beta", "D", "x")))
        given = [s["dy"].float(), torch.zeros_like(x) if s["dx"] is None else s["dx"]]
        grads = torch.autograd.grad([y, x], [leaf[n] for n in names], given)
    t = s["v"].dtype
    out = {"dx0" if n == "x" else "d" + n: d.to(t) if n in ("q", "k", "v") else d for n, d in zip(names, grads)}
    return dict(y=y.detach().to(t), x=x.detach().contiguous(), **out)


def _plain_attend_step(s):
    H, at = s["case"]["heads"], s["slots"].long()
    q, k, v = _heads(s["q"].float(), H), _heads(s["k"].float(), H), s["v"].float()
    kw = k if s["beta"] is None else k * s["beta"].unsqueeze(-1)
    x = torch.exp(s["g"])[..., None, None] * s["x"][at] + kw.unsqueeze(-1) * v.unsqueeze(-2)
    s["x"][at] = x
    y = s["scale"] * (q.unsqueeze(-1) * x).sum(-2)
    if s["D"] is not None:
        y = y + s["D"][:, None] * v
    return dict(y=y.to(s["v"].dtype), x=s["x"])


def _norm_parts(s):
    c = s["case"]
    Bsz, H, L = s["u"].shape
    group = lambda v: v.view(Bsz, c["groups"], H // c["groups"], L)  # noqa: E731
    u, z = s["u"].float(), None if s["z"] is None else s["z"].float()
    p = None if z is None else 1.0 / (1.0 + torch.exp(-z))
    a = group((u * (z * p) if c["gate"] == "before" else u).contiguous())
    if not c["rms"]:
        a = a - a.mean(2, keepdim=True)
    r = 1.0 / torch.sqrt((a * a).mean(2, keepdim=True) + EPS)
    n = (a * r).view(Bsz, H, L)
    pre = n * s["weight"][:, None]
    if s["bias"] is not None:
        pre = pre + s["bias"][:, None]
    return u, z, p, r, n, pre, group


def _plain_norm(s):
    c = s["case"]
    u, z, p, r, n, pre, group = _norm_parts(s)
    y = pre * (z * p) if c["gate"] == "after" else pre
    if c["op"] == "norm":
        return dict(y=y.to(s["u"].dtype))
    t, d, out = s["u"].dtype, s["dy"].float(), dict(y=y.to(s["u"].dtype))
    if c["gate"]:
        slope = p * (1.0 + z * (1.0 - p))
    if c["gate"] == "after":
        out["dz"] = (d * pre * slope).to(t)
        d = d * (z * p)
    # sums over thousands of steps: 64 bits
    out["dweight"] = (d * n).double().sum((0, 2)).float()
    if s["bias"] is not None:
        out["dbias"] = d.double().sum((0, 2)).float()
    dn, ng = group((d * s["weight"][:, None]).contiguous()), group(n)
    da = dn - ng * (dn * ng).mean(2, keepdim=True)
    if not c["rms"]:
        da = da - dn.mean(2, keepdim=True)
    da = (da * r).view(n.shape)
    if c["gate"] == "before":
        out["dz"] = (da * u * slope).to(t)
        da = da * (z * p)
    return dict(du=da.to(t), **out)


_PLAIN = dict(attend=_plain_attend, attend_train=_plain_attend_train, attend_step=_plain_attend_step, norm=_plain_norm,
              norm_train=_plain_norm)


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"].startswith("norm"):
            return _exact_norm(case, s)
        return _exact_step(case, s) if case["op"] == "attend_step" else _exact_attend(case, s)


def _exact_step(case, s):
    f, H, G = torch.float64, case["heads"], case["groups"]
    of = torch.arange(H, device=DEV) // (H // G)
    y, pool = torch.empty(s["v"].shape, dtype=f, device=DEV), s["x"].to(f)
    for b, slot in enumerate(s["slots"].tolist()):
        q, k, v = s["q"][b].to(f)[of], s["k"][b].to(f)[of], s["v"][b].to(f)
        w = torch.ones(H, dtype=f, device=DEV) if s["beta"] is None else s["beta"][b].to(f)
        x = torch.exp(s["g"][b].to(f))[:, None, None] * pool[slot] + torch.einsum("h,hn,hp->hnp", w, k, v)
        pool[slot] = x
        y[b] = s["scale"] * torch.einsum("hn,hnp->hp", q, x)
        if s["D"] is not None:
            y[b] += s["D"].to(f)[:, None] * v
    return dict(y=y, x=pool)


def _exact_attend(case, s):
    """Every pair of a sequence's steps at once, one head at a time."""
    f, H, G, N, P, L = torch.float64, case["heads"], case["groups"], case["keys"], case["values"], case["steps"]
    lens, train = _lengths(case), case["op"] == "attend_train"
    cuts = [0]
    for n in lens:
        cuts.append(cuts[-1] + n)
    spans = [(0, a, b) for a, b in zip(cuts, cuts[1:])] if lens else [(b, 0, L) for b in range(case["batch"])]
    if sum((b - a) ** 2 for _, a, b in spans) * H > 2e10:
        return None
    zeros = lambda v: torch.zeros(v.shape, dtype=f, device=DEV)  # noqa: E731
    y, last = zeros(s["v"]), torch.zeros(len(spans), H, N, P, dtype=f, device=DEV)
    out = {}
    if train:
        out = dict(dq=zeros(s["q"]), dk=zeros(s["k"]), dv=zeros(s["v"]), dg=zeros(s["g"]))
        if s["beta"] is not None:
            out["dbeta"] = zeros(s["beta"])
        if s["D"] is not None:
            out["dD"] = zeros(s["D"])
        if "x" in s:
            out["dx0"] = zeros(s["x"])
    for i, (row, a, b) in enumerate(spans):
        for h in range(H):
            at = h // (H // G)
            Q, K, V = (s[n][row, j, :, a:b].to(f).t() for n, j in (("q", at), ("k", at), ("v", h)))
            Q = Q * s["scale"]
            w = torch.ones(b - a, dtype=f, device=DEV) if s["beta"] is None else s["beta"][row, h, a:b].to(f)
            D = 0.0 if s["D"] is None else s["D"][h].to(f)
            run_ = torch.cumsum(s["g"][row, h, a:b].to(f), 0)
            whole = run_[-1] if b > a else torch.zeros((), dtype=f, device=DEV)
            x0 = s["x"][i, h].to(f) if "x" in s else torch.zeros(N, P, dtype=f, device=DEV)
            fades, keeps = torch.exp(whole - run_), torch.exp(run_)
            last[i, h] = torch.exp(whole) * x0 + (K * (w * fades)[:, None]).t() @ V
            E = (run_[:, None] - run_).masked_fill_(torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).triu_(1), -math.inf)
            E = E.exp_()
            M = (Q @ K.t()).mul_(E)                                   # without beta
            y[row, h, :, a:b] = ((M * w) @ V + D * V + keeps[:, None] * (Q @ x0)).t()
            if not train:
                continue
            dY = s["dy"][row, h, :, a:b].to(f).t()
            dX = torch.zeros(N, P, dtype=f, device=DEV) if s["dx"] is None else s["dx"][i, h].to(f)
            out["dv"][row, h, :, a:b] = ((M * w).t() @ dY + D * dY + (w * fades)[:, None] * (K @ dX)).t()
            dM = dY @ V.t()
            if s["D"] is not None:
                out["dD"][h] += (dY * V).sum()
            EdM = E * dM
            MdM = M.mul_(dM)
            across = fades * ((K @ dX) * V).sum(1)
            if s["beta"] is not None:
                out["dbeta"][row, h, a:b] = MdM.sum(0) + across
            out["dq"][row, at, :, a:b] += (s["scale"] * ((EdM * w) @ K + keeps[:, None] * (dY @ x0.t()))).t()
            out["dk"][row, at, :, a:b] += (w[:, None] * (EdM.t() @ Q + fades[:, None] * (V @ dX.t()))).t()
            MdM *= w
            each = MdM.sum(1) - MdM.sum(0) + keeps * ((Q @ x0) * dY).sum(1) - w * across
            all_ = (w * across).sum() + torch.exp(whole) * (x0 * dX).sum()
            out["dg"][row, h, a:b] = each.flip(0).cumsum(0).flip(0) + all_
            if "x" in s:
                out["dx0"][i, h] = (Q * keeps[:, None]).t() @ dY + torch.exp(whole) * dX
    return dict(y=y, x=last, **out)


def _exact_norm(case, s):
    f, G = torch.float64, case["groups"]
    Bsz, H, L = s["u"].shape
    # steps first: rows of H / G numbers
    rows = lambda v: None if v is None else v.to(f).permute(0, 2, 1).reshape(Bsz * L * G, H // G)  # noqa: E731
    back = lambda v: v.reshape(Bsz, L, H).permute(0, 2, 1)  # noqa: E731
    u, z = rows(s["u"]), rows(s["z"])
    w = s["weight"].to(f).view(G, -1).repeat(Bsz * L, 1)
    b = 0.0 if s["bias"] is None else s["bias"].to(f).view(G, -1).repeat(Bsz * L, 1)
    sig = None if z is None else torch.sigmoid(z)
    a = u * z * sig if case["gate"] == "before" else u
    mu = 0.0 if case["rms"] else a.mean(1, keepdim=True)
    sd = torch.sqrt(((a - mu) ** 2).mean(1, keepdim=True) + EPS)
    n = (a - mu) / sd
    y = n * w + b
    if case["gate"] == "after":
        y = y * z * sig
    if case["op"] == "norm":
        return dict(y=back(y))
    dy = rows(s["dy"])
    out = dict(y=back(y))
    if case["gate"] == "after":
        out["dz"] = back(dy * (n * w + b) * (sig + z * sig * (1 - sig)))
        dy = dy * z * sig
    out["dweight"] = (dy * n).reshape(Bsz * L, H).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dy.reshape(Bsz * L, H).sum(0)
    dn = dy * w
    da = dn - n * (dn * n).mean(1, keepdim=True)
    if not case["rms"]:
        da = da - dn.mean(1, keepdim=True)
    da = da / sd
    if case["gate"] == "before":
        out["dz"] = back(da * u * (sig + z * sig * (1 - sig)))
        da = da * z * sig
    return dict(du=back(da), **out)


# ----------------------------------------------------------------- work ----

def work(case):
    """Each input read once and each output written once; a multiply-add is two operations."""
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    Bsz, L, G = c["batch"], c["steps"], c["groups"]
    if c["op"].startswith("norm"):
        per, H, gate = Bsz * c["channels"] * L, c["channels"], 1 if c["gate"] else 0
        params = 4 * H * (2 if c["bias"] else 1)
        if c["op"] == "norm":
            return dict(bytes=e * per * (2 + gate) + params, flops=per * (6 + 5 * gate))
        # u (and z) in and y out, then u (z) and dy in and du (dz) out
        return dict(bytes=e * per * (5 + 3 * gate) + 3 * params, flops=per * (20 + 15 * gate))
    H, N, P = c["heads"], c["keys"], c["values"]
    T, S = Bsz * L, len(_lengths(c)) or Bsz
    shared, values = e * T * G * N, e * T * H * P
    small = 4 * (T * H if c["decay"] == "token" else H) + (4 * T * H if c["beta"] else 0) + (4 * H if c["skip"] else 0)
    state = 4 * S * H * N * P
    # a step's rank-one update of the state and the product with it
    forward = dict(bytes=2 * shared + 2 * values + small, flops=4 * T * H * N * P)
    if c["op"] == "attend_step":
        return dict(bytes=forward["bytes"] + 2 * state, flops=5 * T * H * N * P)
    forward["bytes"] += state * (2 if c["carry"] else 1)
    if c["op"] == "attend":
        return forward
    # q, k, v, dy, g, beta in and the gradients out; two states walked, three products with them
    back = 4 * shared + 3 * values + 2 * small + (4 * T * H if c["decay"] == "head" else 0) + (3 * state if c["carry"] else 0)
    return dict(bytes=forward["bytes"] + back, flops=14 * T * H * N * P)
