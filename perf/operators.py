"""The selective state-space operators, as cases that can be timed and checked.

Per channel h and state n, with dt = softplus(delta + delta_bias):

    x_t = exp(dt_t A[h,n]) x_{t-1} + dt_t u_t B_t[n]
    y_t = (sum_n C_t[n] x_t[n] + D u_t) * silu(z_t)

and before it the short causal convolution

    y_t = silu(bias + sum_k w[k] u_{t-W+1+k}),   k = 0 .. W-1

for whole prompts (dense, or packed one behind the other), for training (with
every gradient) and for single tokens on states that live in a pool of slots.

`run` computes them in elementary torch operations, in 32 bits, rounded once
at the end; with `own` set it calls the library's entry points.  Activations
are [batch, channels, steps] in either order of storage ("rows": steps
contiguous, "tokens": channels contiguous).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases ----

def _case(name, op, dtype, batch, channels, steps=1, states=0, groups=1, width=0, order="tokens", packed="",
          gate=False, carry=False, pool=0):
    c = dict(op=op, dtype=dtype, batch=batch, channels=channels, steps=steps, states=states, groups=groups,
             width=width, order=order, packed=packed, gate=gate, carry=carry, pool=pool)
    if name:
        c["name"] = name
    return c


def listed():
    prompts = "1,0,517,1300,64,3,2215,996"     # a serving batch: an empty and a one-token prompt, odd lengths
    return [
        # the convolution of one long prompt
        _case("conv long prompt", "conv", "bf16", 1, 4096, 16384, width=4),
        # continued prompts of a serving batch packed one behind the other, on their convolution states
        _case("conv packed prompts", "conv", "f16", 1, 1536, 5096, width=4, packed=prompts, carry=True),
        # gradients of a training batch
        _case("conv gradients", "conv_grad", "bf16", 4, 4096, 2048, width=4),
        # the same in single precision at the filter path's s4-h512-l3k sizes and storage order
        _case("conv gradients rows", "conv_grad", "f32", 16, 512, 3000, width=3, order="rows"),
        # the scan of one long prompt, few channels against its length
        _case("scan long prompt", "scan", "bf16", 1, 2048, 16384, 16, gate=True),
        # continued prompts of a serving batch
        _case("scan packed prompts", "scan", "f16", 1, 4096, 5096, 16, packed=prompts, gate=True, carry=True),
        # a training step: forward with what the backward pass needs, then every gradient
        _case("scan training", "train", "bf16", 4, 4096, 2048, 16, gate=True),
        # the same in single precision at the filter path's s4-h256-l1k sizes and storage order
        _case("scan training rows", "train", "f32", 8, 256, 1024, 64, groups=2, order="rows", carry=True),
        # one sequence's next token: latency
        _case("conv one token", "conv_step", "bf16", 1, 2048, width=4, pool=1),
        # a large decode batch on a pool of slots
        _case("conv decode batch", "conv_step", "f16", 250, 8192, width=4, pool=256),
        _case("scan one token", "step", "bf16", 1, 2048, states=16, gate=True, pool=1),
        _case("scan decode batch", "step", "bf16", 250, 4096, states=16, gate=True, pool=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    return c["batch"] * c["channels"] * c["steps"] * max(1, c["states"])


def draw(rng):
    op = rng.choice(["conv", "conv_grad", "scan", "train", "conv_step", "step"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    most = most // 2 if dtype == "f32" else most
    scan = op in ("scan", "train", "step")
    width = 0 if scan else rng.choice([2, 3, 4])
    while True:
        groups = rng.choice([1, 1, 1, 2, 4]) if scan else 1
        channels = groups * _log_int(rng, 200 // groups, 8192 // groups)
        states = rng.choice([8, 16, 16, 16, 24, 32, 64]) if scan else 0
        gate, carry = scan and rng.random() < 0.6, rng.random() < 0.5
        if op in ("conv_step", "step"):
            batch = _log_int(rng, 1, 256)
            c = _case("", op, dtype, batch, channels, 1, states, groups, width, gate=gate,
                      pool=batch + rng.randrange(1, 17))
        else:
            order = rng.choice(["tokens", "tokens", "rows"])
            steps, batch = _log_int(rng, 100, 16384), _log_int(rng, 1, 16)
            packed = ""
            if op in ("conv", "scan") and rng.random() < 0.4:
                count, batch = rng.randrange(2, 12), 1
                cuts = sorted(rng.randrange(0, steps + 1) for _ in range(count - 1))
                packed = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [steps]))
                order = "tokens"
            if op == "conv_grad":
                carry = False
            c = _case("", op, dtype, batch, channels, steps, states, groups, width, order, packed, gate, carry)
        if _cost(c) <= most:
            return c


# --------------------------------------------------------------- inputs ----

def _lengths(c):
    return [int(v) for v in c["packed"].split(",")] if c["packed"] else []


def prepare(case, seed):
    c, t = case, DTYPES[case["dtype"]]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    Bsz, H, L, N, G, W = (c[k] for k in ("batch", "channels", "steps", "states", "groups", "width"))

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=DEV) * scale

    def act(*shape, scale=1.0):
        # [batch, ..., steps] of the activations' type; in "tokens" order the steps' axis is stored first
        if c["order"] == "tokens" and len(shape) > 2:
            return normal(shape[0], shape[-1], *shape[1:-1], scale=scale).to(t).movedim(1, -1)
        return normal(*shape, scale=scale).to(t)

    single = c["op"] in ("conv_step", "step")
    time = () if single else (L,)
    s = dict(case=case, u=act(Bsz, H, *time))
    lens = _lengths(c)
    S = len(lens) if lens else Bsz
    if lens:
        offs = [0]
        for n in lens:
            offs.append(offs[-1] + n)
        s["offsets"] = torch.tensor(offs, dtype=torch.int32, device=DEV)
        # the plan of the packed batch: each token's sequence and place in it
        seq = torch.repeat_interleave(torch.arange(S, device=DEV), torch.tensor(lens, device=DEV))
        s["seq"] = seq
        s["pos"] = torch.arange(L, device=DEV) - s["offsets"].long()[seq]
        s["live"] = torch.tensor([i for i, n in enumerate(lens) if n], device=DEV)
    if c["pool"]:
        s["slots"] = torch.randperm(c["pool"], generator=g, device=DEV)[:Bsz].to(torch.int32)
    if W:
        s["weight"] = normal(H, W, scale=1.0 / math.sqrt(W))
        s["bias"] = normal(H, scale=0.1)
        if single:
            s["state"] = normal(c["pool"], H, W - 1).to(t)
        elif c["carry"]:
            s["state"] = normal(S, H, W - 1).to(t)
    else:
        s["delta"] = act(Bsz, H, *time, scale=0.7)
        # step sizes log-uniform in [1e-3, 1e-1] at delta = 0
        lo, hi = math.log(1e-3), math.log(1e-1)
        dt = torch.exp(lo + (hi - lo) * torch.rand(H, generator=g, device=DEV))
        s["delta_bias"] = dt + torch.log(-torch.expm1(-dt))
        s["A"] = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(normal(H, N, scale=0.1))
        s["B"], s["C"] = act(Bsz, G, N, *time), act(Bsz, G, N, *time)
        s["D"] = 1.0 + normal(H, scale=0.1)
        s["z"] = act(Bsz, H, *time) if c["gate"] else None
        if single:
            s["x"] = normal(c["pool"], H, N, scale=0.3)
        elif c["carry"]:
            s["x"] = normal(S, H, N, scale=0.3)
    if c["op"] in ("conv_grad", "train"):
        s["dy"] = act(Bsz, H, L)
    return s


# ------------------------------------------------- the library's calls ----

def _run_own(s):
    from structured_state_space_amd import ssm
    op = s["case"]["op"]
    if op == "conv":
        st = s.get("state")
        out = ssm.causal_conv(s["u"], s["weight"], s["bias"], silu=True, state=st, want_state=True,
                              offsets=s.get("offsets"))
        return dict(y=out["y"], state=out["state"])
    if op == "conv_grad":
        return ssm.causal_conv_backward(s["u"], s["weight"], s["dy"], s["bias"], silu=True)
    if op == "conv_step":
        out = ssm.causal_conv_step(s["u"], s["weight"], s["state"], s["bias"], silu=True, slots=s["slots"])
        return dict(y=out["y"], state=out["state"])
    if op == "step":
        out = ssm.selective_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["x"], D=s["D"], z=s["z"],
                                 delta_bias=s["delta_bias"], softplus=True, slots=s["slots"])
        return dict(y=out["y"], x=out["x"])
    args = (s["u"], s["delta"], s["A"], s["B"], s["C"])
    more = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=True, x0=s.get("x"))
    if op == "scan":
        out = ssm.selective_scan(*args, want_state=True, offsets=s.get("offsets"), **more)
        return dict(y=out["y"], x=out["x"])
    out = ssm.selective_scan(*args, want_state=True, save=True, **more)
    grads = ssm.selective_scan_backward(*args, s["dy"], saved=out["saved"], **more)
    return dict(y=out["y"], x=out["x"], **{k: v for k, v in grads.items() if v is not None})


# ------------------------------------------------------ the plain forms ----

def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _silu_slope(v):
    p = 1.0 / (1.0 + torch.exp(-v))
    return p * (1.0 + v * (1.0 - p))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _history(s, u, state):
    """The W inputs under the kernel at each step: W tensors like u, oldest first."""
    W, L = s["case"]["width"], u.shape[-1]
    if "seq" not in s:
        past = u.new_zeros(u.shape[0], u.shape[1], W - 1) if state is None else state
        full = torch.cat([past, u], -1)
        return [full[..., k:k + L] for k in range(W)]
    taps = []
    for k in range(W):
        back = W - 1 - k
        at = torch.arange(L, device=u.device)
        v = u[..., torch.clamp(at - back, min=0)]
        old = torch.clamp(W - 1 + s["pos"] - back, max=W - 2)
        past = u.new_zeros(()) if state is None else state[s["seq"], :, old].t().unsqueeze(0)
        taps.append(torch.where(s["pos"] >= back, v, past))
    return taps


def _last_inputs(s, u, state):
    """The last W - 1 inputs of every sequence, oldest first."""
    W = s["case"]["width"]
    if "seq" not in s:
        past = u.new_zeros(u.shape[0], u.shape[1], W - 1) if state is None else state
        return torch.cat([past, u], -1)[..., -(W - 1):]
    begin, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    cols = []
    for j in range(W - 1):
        at = end - (W - 1) + j
        v = u[0][:, torch.clamp(at, min=0)].t()
        old = torch.clamp(end - begin + j, max=W - 2)
        past = u.new_zeros(()) if state is None else state[torch.arange(len(end), device=u.device), :, old]
        cols.append(torch.where((at >= begin).unsqueeze(1), v, past))
    return torch.stack(cols, -1)


def _plain_conv(s):
    u = s["u"].float()
    state = s["state"].float() if s.get("state") is not None else None
    pre = s["bias"][:, None]
    for k, v in enumerate(_history(s, u, state)):
        pre = pre + s["weight"][:, k, None] * v
    t = s["u"].dtype
    return dict(y=_silu(pre).to(t), state=_last_inputs(s, u, state).to(t))


def _plain_conv_grad(s):
    u, dy, w, W, L = s["u"].float(), s["dy"].float(), s["weight"], s["case"]["width"], s["case"]["steps"]
    taps = _history(s, u, None)
    pre = s["bias"][:, None]
    for k, v in enumerate(taps):
        pre = pre + w[:, k, None] * v
    dpre = dy * _silu_slope(pre)
    ahead = torch.cat([dpre, dpre.new_zeros(*dpre.shape[:2], W - 1)], -1)
    du = sum(w[:, k, None] * ahead[..., W - 1 - k:W - 1 - k + L] for k in range(W))
    # sums over the batch and thousands of steps: 64 bits
    dw = torch.stack([(dpre * v).double().sum((0, 2)) for v in taps], 1)
    return dict(du=du.to(s["u"].dtype), dweight=dw.float(), dbias=dpre.double().sum((0, 2)).float())


def _plain_conv_step(s):
    at = s["slots"].long()
    full = torch.cat([s["state"][at].float(), s["u"].float().unsqueeze(-1)], -1)
    y = _silu(s["bias"] + (s["weight"] * full).sum(-1)).to(s["u"].dtype)
    s["state"][at] = full[..., 1:].to(s["state"].dtype)
    return dict(y=y, state=s["state"])


def _recur(a, b):
    """x_t = a_t x_{t-1} + b_t along the last axis (x_{-1} = 0), by doubling: log2(steps) passes; both are overwritten."""
    d = 1
    while d < b.shape[-1]:
        b[..., d:] += a[..., d:] * b[..., :-d]
        a[..., d:] = a[..., d:] * a[..., :-d]
        d *= 2
    return b


def _spread(v, H):
    """[batch, groups, ...] -> [batch, channels, ...]"""
    return v.repeat_interleave(H // v.shape[1], 1)


def _forward(s):
    """dt, the decays, the states at every step and the ungated output, in 32 bits."""
    H = s["case"]["channels"]
    u, dt = s["u"].float(), _softplus(s["delta"].float() + s["delta_bias"][:, None])
    B, C = _spread(s["B"].float(), H), _spread(s["C"].float(), H)
    decay = torch.exp(dt.unsqueeze(2) * s["A"].unsqueeze(-1))
    b = (dt * u).unsqueeze(2) * B
    a = decay.clone()
    x0 = s.get("x")
    if "seq" not in s:
        if x0 is not None:
            b[..., 0] += a[..., 0] * x0
        x = _recur(a, b)
        last = x[..., -1]
    else:
        live, offs = s["live"], s["offsets"].long()
        starts = offs[:-1][live]
        if x0 is not None:
            b[0][:, :, starts] += a[0][:, :, starts] * x0[live].permute(1, 2, 0)
        a[0][:, :, starts] = 0.0
        x = _recur(a, b)
        last = x.new_zeros(len(offs) - 1, *x.shape[1:3]) if x0 is None else x0.clone()
        last[live] = x[0][:, :, offs[1:][live] - 1].permute(2, 0, 1)
    pre = (C * x).sum(2) + s["D"][:, None] * u
    return u, dt, B, C, decay, x, pre, last


def _plain_scan(s):
    _, _, _, _, _, _, pre, last = _forward(s)
    y = pre * _silu(s["z"].float()) if s["z"] is not None else pre
    return dict(y=y.to(s["u"].dtype), x=last.clone())


def _plain_train(s):
    H, t = s["case"]["channels"], s["u"].dtype
    u, dt, B, C, decay, x, pre, last = _forward(s)
    dpre, out = s["dy"].float(), {}
    y = pre
    if s["z"] is not None:
        z = s["z"].float()
        y = pre * _silu(z)
        out["dz"] = (dpre * pre * _silu_slope(z)).to(t)
        dpre = dpre * _silu(z)
    G = s["B"].shape[1]

    def by_group(v):
        return v.reshape(v.shape[0], G, H // G, *v.shape[2:]).sum(2)

    out["dC"] = by_group(dpre.unsqueeze(2) * x).to(t)
    # from here on x is the state before each step
    x0 = s.get("x")
    first = torch.zeros_like(last) if x0 is None else x0
    x = torch.cat([first.unsqueeze(-1), x[..., :-1]], -1)
    # g_t = C_t dpre_t + decay_{t+1} g_{t+1}: the same recurrence from the end
    later = torch.cat([decay[..., 1:], torch.zeros_like(decay[..., :1])], -1).flip(-1)
    g = _recur(later, (C * dpre.unsqueeze(2)).flip(-1)).flip(-1)
    out["dB"] = by_group(g * (dt * u).unsqueeze(2)).to(t)
    gB = (g * B).sum(2)
    if x0 is not None:
        out["dx0"] = decay[..., 0] * g[..., 0]
    back = g * x * decay
    slope = -torch.expm1(-dt)                             # the slope of softplus: sigmoid(v) = 1 - exp(-softplus(v))
    ddelta = ((back * s["A"].unsqueeze(-1)).sum(2) + u * gB) * slope
    # sums over the batch and thousands of steps: 64 bits
    out["dA"] = (back * dt.unsqueeze(2)).double().sum((0, 3)).float()
    out["dD"] = (dpre * u).double().sum((0, 2)).float()
    out["ddelta_bias"] = ddelta.double().sum((0, 2)).float()
    out["du"] = (s["D"][:, None] * dpre + dt * gB).to(t)
    out["ddelta"] = ddelta.to(t)
    return dict(y=y.to(t), x=last.clone(), **out)


def _plain_step(s):
    H, at = s["case"]["channels"], s["slots"].long()
    u, dt = s["u"].float(), _softplus(s["delta"].float() + s["delta_bias"])
    B, C = _spread(s["B"].float(), H), _spread(s["C"].float(), H)
    x = torch.exp(dt.unsqueeze(-1) * s["A"]) * s["x"][at] + (dt * u).unsqueeze(-1) * B
    s["x"][at] = x
    y = (C * x).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return dict(y=y.to(s["u"].dtype), x=s["x"])


_PLAIN = dict(conv=_plain_conv, conv_grad=_plain_conv_grad, conv_step=_plain_conv_step, scan=_plain_scan,
              train=_plain_train, step=_plain_step)


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return (_exact_conv if case["width"] else _exact_scan)(case, s)


def _segments(case):
    """(row, begin, end, sequence) of every sequence."""
    lens, at, out = _lengths(case), 0, []
    for i, n in enumerate(lens):
        out.append((0, at, at + n, i))
        at += n
    return out or [(b, 0, case["steps"], b) for b in range(case["batch"])]


def _exact_conv(case, s):
    W, f = case["width"], torch.float64
    w, bias = s["weight"].to(f), s["bias"].to(f)
    if case["op"] == "conv_step":
        state = s["state"].clone()
        y = torch.empty(s["u"].shape, dtype=f, device=DEV)
        for b, slot in enumerate(s["slots"].tolist()):
            line = torch.cat([state[slot].to(f), s["u"][b].to(f)[:, None]], 1)
            pre = (line * w).sum(1) + bias
            y[b] = pre * torch.sigmoid(pre)
            state[slot] = line[:, 1:].to(state.dtype)
        return dict(y=y, state=state.to(f))
    u = s["u"].to(f)
    if case["op"] == "conv":
        y, ends = torch.empty(u.shape, dtype=f, device=DEV), []
        for row, begin, end, i in _segments(case):
            past = s["state"][i].to(f) if "state" in s else torch.zeros(u.shape[1], W - 1, dtype=f, device=DEV)
            line = torch.cat([past, u[row, :, begin:end]], 1)
            if end > begin:
                pre = torch.einsum("hlk,hk->hl", line.unfold(1, W, 1), w) + bias[:, None]
                y[row, :, begin:end] = pre * torch.sigmoid(pre)
            ends.append(line[:, line.shape[1] - (W - 1):])
        return dict(y=y, state=torch.stack(ends))
    dw, db, du = torch.zeros_like(w), torch.zeros_like(bias), torch.empty(u.shape, dtype=f, device=DEV)
    for b in range(u.shape[0]):
        line = torch.nn.functional.pad(u[b], (W - 1, 0))
        pre = bias[:, None] + sum(w[:, k:k + 1] * line[:, k:k + u.shape[2]] for k in range(W))
        p = torch.sigmoid(pre)
        d = s["dy"][b].to(f) * (p + pre * p * (1 - p))
        dline = torch.zeros_like(line)
        for k in range(W):
            dw[:, k] += (d * line[:, k:k + u.shape[2]]).sum(1)
            dline[:, k:k + u.shape[2]] += w[:, k:k + 1] * d
        db += d.sum(1)
        du[b] = dline[:, W - 1:]
    return dict(du=du, dweight=dw, dbias=db)


def _exact_scan(case, s):
    f, H, N, G = torch.float64, case["channels"], case["states"], case["groups"]
    if case["steps"] * (2 if case["op"] == "train" else 1) > 70000:
        return None
    A, D, bias = s["A"].to(f), s["D"].to(f), s["delta_bias"].to(f)
    of = torch.arange(H, device=DEV) // (H // G)
    softplus = lambda v: torch.logaddexp(v, torch.zeros_like(v))  # noqa: E731
    if case["op"] == "step":
        at = s["slots"].long()
        u, dt = s["u"].to(f), softplus(s["delta"].to(f) + bias)
        pool = s["x"].to(f)
        x = torch.exp(dt[..., None] * A) * pool[at] + (dt * u)[..., None] * s["B"].to(f)[:, of]
        pool[at] = x
        y = torch.einsum("bhn,bhn->bh", x, s["C"].to(f)[:, of]) + D * u
        if s["z"] is not None:
            y = y * s["z"].to(f) * torch.sigmoid(s["z"].to(f))
        return dict(y=y, x=pool)
    L, Bsz, train = case["steps"], case["batch"], case["op"] == "train"
    # steps first, so that one step is one contiguous slice
    u, z, delta = (s[k].to(f).permute(2, 0, 1).contiguous() if s[k] is not None else None for k in ("u", "z", "delta"))
    Bt, Ct = (s[k].permute(3, 0, 1, 2).contiguous() for k in ("B", "C"))
    dt = softplus(delta + bias)
    pre = torch.empty_like(u)
    x0 = s["x"].to(f) if "x" in s else torch.zeros(len(_lengths(case)) or Bsz, H, N, dtype=f, device=DEV)
    last, states = x0.clone(), (torch.empty(L + 1, Bsz, H, N, dtype=f, device=DEV) if train else None)
    spans = _segments(case) if case["packed"] else [(slice(None), 0, L, slice(None))]
    for _, begin, end, i in spans:
        x = x0[i].reshape(-1, H, N) if case["packed"] else x0
        if train:
            states[0] = x
        for t in range(begin, end):
            x = torch.exp(dt[t, :, :, None] * A) * x + (dt[t] * u[t])[..., None] * Bt[t].to(f)[:, of]
            pre[t] = (x * Ct[t].to(f)[:, of]).sum(-1) + D * u[t]
            if train:
                states[t + 1] = x
        last[i] = x
    y = pre * z * torch.sigmoid(z) if z is not None else pre
    if not train:
        return dict(y=y.permute(1, 2, 0), x=last)
    dy, out = s["dy"].to(f).permute(2, 0, 1).contiguous(), {}
    dpre = dy
    if z is not None:
        p = torch.sigmoid(z)
        out["dz"] = (dy * pre * (p + z * p * (1 - p))).permute(1, 2, 0)
        dpre = dy * z * p
    du, ddt, dA, carry = D * dpre, torch.empty_like(dt), torch.zeros_like(A), torch.zeros_like(x0)
    dB, dC = torch.zeros(L, Bsz, G, N, dtype=f, device=DEV), torch.zeros(L, Bsz, G, N, dtype=f, device=DEV)
    for t in range(L - 1, -1, -1):
        g = carry + dpre[t, :, :, None] * Ct[t].to(f)[:, of]
        dC[t] = (dpre[t, :, :, None] * states[t + 1]).view(Bsz, G, H // G, N).sum(2)
        dB[t] = (g * (dt[t] * u[t])[..., None]).view(Bsz, G, H // G, N).sum(2)
        gB = (g * Bt[t].to(f)[:, of]).sum(-1)
        carry = g * torch.exp(dt[t, :, :, None] * A)
        back = carry * states[t]
        ddt[t] = (back * A).sum(-1) + u[t] * gB
        dA += (back * dt[t, :, :, None]).sum(0)
        du[t] += dt[t] * gB
    ddelta = ddt * torch.sigmoid(delta + bias)
    if "x" in s:
        out["dx0"] = carry
    out.update(dA=dA, dB=dB.permute(1, 2, 3, 0), dC=dC.permute(1, 2, 3, 0), dD=(dpre * u).sum((0, 1)),
               ddelta_bias=ddelta.sum((0, 1)), du=du.permute(1, 2, 0), ddelta=ddelta.permute(1, 2, 0))
    return dict(y=y.permute(1, 2, 0), x=last, **out)


# ----------------------------------------------------------------- work ----

def work(case):
    """Each input read once and each output written once; a multiply-add is two operations."""
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    Bsz, H, L, N, G, W = (c[k] for k in ("batch", "channels", "steps", "states", "groups", "width"))
    per, S = Bsz * H * L, len(_lengths(c)) or Bsz
    if c["op"] == "conv":
        return dict(bytes=2 * e * per + 4 * H * (W + 1) + e * S * H * (W - 1) * (2 if c["carry"] else 1),
                    flops=per * (2 * W + 5))
    if c["op"] == "conv_grad":
        return dict(bytes=3 * e * per + 8 * H * (W + 1), flops=per * (6 * W + 12))
    if c["op"] == "conv_step":
        return dict(bytes=2 * e * per + 2 * e * per * (W - 1) + 4 * H * (W + 1), flops=per * (2 * W + 5))
    acts, shared = (4 if c["gate"] else 3) * e * per, 2 * e * Bsz * G * N * L
    params = 4 * H * (N + 2)
    if c["op"] == "step":
        return dict(bytes=acts + shared + params + 8 * per * N, flops=per * (7 * N + 16))
    state = 4 * S * H * N * (2 if c["carry"] else 1)
    if c["op"] == "scan":
        return dict(bytes=acts + shared + params + state, flops=per * (7 * N + 16))
    # the forward pass, then u, delta, z, dy, B, C in and du, ddelta, dz, dB, dC out
    back = (7 if c["gate"] else 5) * e * per + 2 * shared + 2 * params + (2 * 4 * S * H * N if c["carry"] else 0)
    return dict(bytes=acts + shared + params + state + back, flops=per * (22 * N + 60))
