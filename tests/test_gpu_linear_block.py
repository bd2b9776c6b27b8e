"""The operators as a layer uses them: short convolution, linear attention on its
slices, gated norm. Training through torch.autograd.Function, prompts then tokens on
pools of states, both captured into graphs, against a plain float64 layer."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"
H, G, N, P, W = 4, 2, 32, 16, 4
C = H * P + 2 * G * N          # channels of the convolution
SCALE = N ** -0.5


def _ssm():
    from structured_state_space_amd import ssm
    return ssm


def _weights(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return dict(w=0.5 * r(C, W), b=0.1 * r(C), D=r(H), rate=1.0 + torch.rand(H, generator=g, device=DEV), norm=1.0 + 0.2 * r(H * P),
                dt_bias=-2.0 + 0.3 * r(H))


def _slices(u):
    """v, k, q of the convolution's output [Bsz, C, L] (or [Bsz, C])"""
    v, k, q = u[:, :H * P], u[:, H * P:H * P + G * N], u[:, H * P + G * N:]
    return v.unflatten(1, (H, P)), k.unflatten(1, (G, N)), q.unflatten(1, (G, N))


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, w, b):
        ctx.save_for_backward(u, w, b)
        return _ssm().causal_conv(u, w, b, silu=True)["y"]

    @staticmethod
    def backward(ctx, dy):
        u, w, b = ctx.saved_tensors
        g = _ssm().causal_conv_backward(u, w, dy, b, silu=True)
        return g["du"], g["dweight"], g["dbias"]


class Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, D):
        f = _ssm().linear_attention(q, k, v, g, beta=beta, D=D, scale=SCALE, save=True)
        ctx.save_for_backward(q, k, v, g, beta, D, f["saved"])
        return f["y"]

    @staticmethod
    def backward(ctx, dy):
        q, k, v, g, beta, D, saved = ctx.saved_tensors
        d = _ssm().linear_attention_backward(q, k, v, g, dy, beta=beta, D=D, scale=SCALE, saved=saved)
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], d["dD"]


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, z, w):
        ctx.save_for_backward(u, z, w)
        return _ssm().layer_norm(u, w, z=z, gate="before", rms=True, groups=G)["y"]

    @staticmethod
    def backward(ctx, dy):
        u, z, w = ctx.saved_tensors
        g = _ssm().layer_norm_backward(u, dy, w, z=z, gate="before", rms=True, groups=G)
        return g["du"], g["dz"], g["dweight"]


def layer(x, z, dt, p):
    """x [Bsz, C, L], z [Bsz, H P, L], dt [Bsz, H, L] float32 -> [Bsz, H P, L]"""
    u = Conv.apply(x, p["w"], p["b"])
    v, k, q = _slices(u)
    step = torch.nn.functional.softplus(dt + p["dt_bias"][:, None])
    y = Attend.apply(q, k, v, -step * p["rate"][:, None], step, p["D"])
    return Norm.apply(y.flatten(1, 2), z, p["norm"])


def plain(x, z, dt, p):
    """The same in float64, step by step, for autograd."""
    Bsz, _, L = x.shape
    line = torch.nn.functional.pad(x, (W - 1, 0))
    u = torch.nn.functional.silu(sum(line[..., i:i + L] * p["w"][:, i:i + 1] for i in range(W)) + p["b"][:, None])
    v, k, q = _slices(u)
    k, q = (t.repeat_interleave(H // G, 1) for t in (k, q))
    step = torch.nn.functional.softplus(dt + p["dt_bias"][:, None])
    state, ys = x.new_zeros((Bsz, H, N, P)), []
    for t in range(L):
        e = torch.exp(-step[..., t] * p["rate"])
        state = e[..., None, None] * state + (step[..., t, None] * k[..., t])[..., None] * v[..., t][:, :, None]
        ys.append(SCALE * (q[..., t][..., None] * state).sum(2) + p["D"][:, None] * v[..., t])
    a = (torch.stack(ys, -1).flatten(1, 2) * torch.nn.functional.silu(z)).unflatten(1, (G, -1))
    n = a / torch.sqrt((a * a).mean(2, keepdim=True) + 1e-5)
    return n.flatten(1, 2) * p["norm"][:, None]


def _inputs(seed, Bsz, L, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda c: torch.randn((Bsz, L, c), generator=g, device=DEV)  # noqa: E731
    return r(C).to(dtype).transpose(1, 2), r(H * P).to(dtype).transpose(1, 2), r(H).transpose(1, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_step(dtype):
    """Forward and every gradient of the layer against the plain one.  The layer's activations are rounded
    three times on the way (by half a step each) and as often back: in norm six half steps, twice that allowed;
    float32: 1e-5 of the norm, some hundred half steps."""
    p = _weights(1)
    x, z, dt = _inputs(2, 2, 150, dtype)
    leaves = [t.detach().clone().requires_grad_() for t in (x, z, dt, *p.values())]
    y = layer(*leaves[:3], dict(zip(p, leaves[3:])))
    dy = torch.randn(y.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(dtype)
    y.backward(dy)
    wide = [t.detach().double().cpu().requires_grad_() for t in leaves]
    want = plain(*wide[:3], dict(zip(p, wide[3:])))
    want.backward(dy.double().cpu())
    tol = 1e-5 if dtype == torch.float32 else 12 * 2.0 ** -8
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(y.detach(), want.detach()) <= tol
    for n, a, b in zip(["x", "z", "dt", *p], leaves, wide):
        assert rel(a.grad, b.grad) <= tol, n


def test_captured_training_step():
    """Forward and backward in one graph, replayed with new inputs between eager calls: every replay equals the
    eager result."""
    ssm = _ssm()
    p = _weights(4)
    x, z, dt = (t.clone(memory_format=torch.preserve_format) for t in _inputs(5, 2, 200, torch.bfloat16))
    dy = torch.randn_like(z)

    def step():
        u = ssm.causal_conv(x, p["w"], p["b"], silu=True)["y"]
        v, k, q = _slices(u)
        s = torch.nn.functional.softplus(dt + p["dt_bias"][:, None])
        g = -s * p["rate"][:, None]
        f = ssm.linear_attention(q, k, v, g, beta=s, D=p["D"], scale=SCALE, save=True, want_state=True)
        a = f["y"].flatten(1, 2)
        n = ssm.layer_norm(a, p["norm"], z=z, gate="before", rms=True, groups=G)["y"]
        gn = ssm.layer_norm_backward(a, dy, p["norm"], z=z, gate="before", rms=True, groups=G)
        ga = ssm.linear_attention_backward(q, k, v, g, gn["du"].unflatten(1, (H, P)), beta=s, D=p["D"], scale=SCALE,
                                           saved=f["saved"])
        return [t for t in (n, f["x"], *gn.values(), *ga.values()) if t is not None]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    gen = torch.Generator(device=DEV).manual_seed(6)
    for _ in range(4):
        for t in (x, z, dt, dy):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompts_then_tokens(dtype):
    """Packed prompts on pools of states, then tokens one by one, against the plain layer on the whole
    sequences (tolerances as above, forward only)."""
    ssm = _ssm()
    p = _weights(7)
    lens, more = [37, 1, 90], 6
    full = [_inputs(8 + i, 1, n + more, dtype) for i, n in enumerate(lens)]
    packed = [torch.cat([f[j][..., :n] for f, n in zip(full, lens)], -1) for j in range(3)]
    offsets = torch.tensor([0, 37, 38, 128], dtype=torch.int32, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    conv, pool = torch.zeros((5, C, W - 1), dtype=dtype, device=DEV), torch.zeros((5, H, N, P), device=DEV)
    x, z, dt = packed
    u = ssm.causal_conv(x, p["w"], p["b"], silu=True, state=conv, state_out=conv, offsets=offsets, slots=slots)["y"]
    v, k, q = _slices(u)
    s = torch.nn.functional.softplus(dt + p["dt_bias"][:, None])
    a = ssm.linear_attention(q, k, v, -s * p["rate"][:, None], beta=s, D=p["D"], scale=SCALE, x0=pool, x_out=pool, offsets=offsets,
                             slots=slots)["y"]
    y = ssm.layer_norm(a.flatten(1, 2), p["norm"], z=z, gate="before", rms=True, groups=G)["y"]
    tokens = []
    for t in range(more):
        x, z, dt = (torch.cat([f[j][..., n + t] for f, n in zip(full, lens)]) for j in range(3))
        u = ssm.causal_conv_step(x, p["w"], conv, p["b"], silu=True, slots=slots)["y"]
        v, k, q = _slices(u)
        s = torch.nn.functional.softplus(dt + p["dt_bias"])
        a = ssm.linear_attention_step(q, k, v, -s * p["rate"], pool, beta=s, D=p["D"], scale=SCALE, slots=slots)["y"]
        tokens.append(ssm.layer_norm(a.flatten(1), p["norm"], z=z, gate="before", rms=True, groups=G)["y"])
    tol = 1e-5 if dtype == torch.float32 else 6 * 2.0 ** -8
    for i, n in enumerate(lens):
        want = plain(*(f.double().cpu() for f in full[i]), {m: w.double().cpu() for m, w in p.items()})[0]
        got = torch.cat([y[0, :, int(offsets[i]):int(offsets[i + 1])], torch.stack([t[i] for t in tokens], -1)], -1).double().cpu()
        assert float((got - want).norm() / want.norm()) <= tol
