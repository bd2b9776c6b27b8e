"""Layer norm at sizes where a launch or an index could end."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"


def _ssm():
    from structured_state_space_amd import ssm
    return ssm


def test_more_than_2_to_22_rows_of_tokens():
    """Flattened tokens with a norm for each head: 2^22 (token, group) rows, as one token each and as steps of a batch
    (the same kernel on the same rows: the same bits)."""
    ssm = _ssm()
    Bsz, H, G = 1 << 16, 2048, 64
    gen = torch.Generator(device=DEV).manual_seed(1)
    u, z, dy = (torch.randn((Bsz, H), generator=gen, device=DEV).bfloat16() for _ in range(3))
    w = torch.randn(H, generator=gen, device=DEV)
    more = dict(weight=w, gate="before", rms=True, groups=G)
    y = ssm.layer_norm(u, z=z, **more)["y"]
    g = ssm.layer_norm_backward(u, dy, z=z, **more)
    steps = lambda t: t.view(16, Bsz // 16, H).transpose(1, 2)  # noqa: E731
    want = ssm.layer_norm(steps(u), z=steps(z), **more)["y"]
    back = ssm.layer_norm_backward(steps(u), steps(dy), z=steps(z), **more)
    assert torch.equal(steps(y), want)
    assert all(torch.equal(steps(g[k]), back[k]) for k in ("du", "dz")) and torch.equal(g["dweight"], back["dweight"])


def test_gradients_of_2_to_27_parameters():
    """The parameters' sums in more units of sixteen channels than a launch of one each has threads for."""
    ssm = _ssm()
    H, G = (1 << 27) + 1024, (1 << 21) + 16
    gen = torch.Generator(device=DEV).manual_seed(2)
    u, dy = (torch.randn((1, H), generator=gen, device=DEV).bfloat16() for _ in range(2))
    w = torch.ones(H, device=DEV)
    g = ssm.layer_norm_backward(u, dy, weight=w, bias=w, groups=G)
    for i in (0, G // 2, G - 1):
        at = slice(64 * i, 64 * i + 64)
        part = ssm.layer_norm_backward(u[:, at].contiguous(), dy[:, at].contiguous(), weight=w[at], bias=w[at])
        assert torch.equal(g["du"][:, at], part["du"])
        assert torch.equal(g["dweight"][at], part["dweight"]) and torch.equal(g["dbias"][at], part["dbias"])


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("order", ["tokens", "rows"])
def test_variances_below_the_normal_numbers(order, rms):
    """eps of zero and inputs of 1e-20: the mean square is a subnormal number of float32, whose root is not zero.
    Squares are rounded to multiples of 2^-149, half of one each, and so is their mean: (1 + 1/2) 2^-150 of it, half
    of that relative to the root; 200 half steps for all else, as in the norm's other tests."""
    import oracle.linear_oracle as O
    from tests.selective_cases import on_device, rounded
    ssm = _ssm()
    D = 48
    u = rounded(np.random.default_rng(3).standard_normal((2, D, 9)) * 1e-20, "f32")
    got = ssm.layer_norm(on_device(u, "f32", order), rms=rms, eps=0.0)["y"].double().cpu().numpy()
    want, _, r = O.norm(u, None, None, None, "after", rms, 1, 0.0)
    square = 1.0 / r[:, 0] ** 2
    tol = np.abs(want) * (1.5 * 2.0 ** -150 / square / 2.0) + 200.0 * 2.0 ** -24 * (np.abs(want) + 1.0)
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
