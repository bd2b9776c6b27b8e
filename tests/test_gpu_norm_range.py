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
