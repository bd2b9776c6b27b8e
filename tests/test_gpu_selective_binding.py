"""What the binding of the selective operators makes of unusual but allowed
arguments, and how it refuses wrong ones."""
import pytest

from tests.test_gpu_selective import DEV, _int, _ssm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _random(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device=DEV)


def test_slots_without_states():
    """Without a state array a slot only says whether its sequence runs: any number
    from 0 on does, a negative one does not, as in the calls with a pool beside them."""
    ssm, r = _ssm(), _random(71)
    slots, run = _int([9, -1, 4, 2**20]), [0, 2, 3]
    u, w, A = r(4, 12, 20), r(12, 4), -torch.rand((12, 16), device=DEV)
    B, C, x = r(4, 1, 16, 20), r(4, 1, 16, 20), r(4, 12, 20)

    def check(got, want):
        assert torch.equal(got[run], want[run]) and bool((got[1] == 7.0).all())

    for width in (1, 4):
        y = torch.full_like(u, 7.0)
        check(ssm.causal_conv(u, w[:, :width].contiguous(), slots=slots, y=y)["y"],
              ssm.causal_conv(u, w[:, :width].contiguous())["y"])
    y = torch.full_like(u, 7.0)
    check(ssm.selective_scan(u, x, A, B, C, softplus=True, slots=slots, y=y)["y"],
          ssm.selective_scan(u, x, A, B, C, softplus=True)["y"])
    y = torch.full((4, 12), 7.0, device=DEV)
    t = u[..., 0].contiguous()
    check(ssm.causal_conv_step(t, w[:, :1].contiguous(), None, slots=slots, y=y)["y"],
          ssm.causal_conv_step(t, w[:, :1].contiguous(), None)["y"])


def test_refusals_name_the_argument():
    ssm, r = _ssm(), _random(72)
    u, w, A = r(1, 8, 20), r(8, 4), -torch.rand((8, 16), device=DEV)
    B = r(1, 1, 16, 20)
    scan = lambda **kw: ssm.selective_scan(u, u, A, B, B, **kw)  # noqa: E731
    back = lambda **kw: ssm.selective_scan_backward(u, u, A, B, B, u, **kw)  # noqa: E731
    conv = lambda **kw: ssm.causal_conv(u, w, **kw)  # noqa: E731
    none = torch.empty((0, 8, 16), device=DEV), torch.empty((0, 8, 3), device=DEV)
    for call, kw, name in [
        (scan, dict(offsets=[0, 20]), "offsets"), (conv, dict(offsets=[0, 20]), "offsets"),
        (scan, dict(offsets=torch.tensor(20, dtype=torch.int32, device=DEV)), "offsets"),
        (conv, dict(offsets=_int([20])), "offsets"), (back, dict(offsets=[0, 20]), "offsets"),
        (scan, dict(offsets=torch.tensor([0, 20], device=DEV)), "offsets"),      # int64
        (scan, dict(x0=0.0), "x0"), (back, dict(x0=0.0), "x0"), (scan, dict(x_out=1), "x_out"),
        (conv, dict(state=0.0), "state"), (scan, dict(lengths=[20]), "lengths"), (scan, dict(slots=[0]), "slots"),
        # a pool without rows
        (scan, dict(x0=none[0], x_out=none[0], slots=_int([0])), "x0"),
        (scan, dict(x_out=none[0], slots=_int([0])), "x_out"),
        (conv, dict(state=none[1], state_out=none[1], slots=_int([0])), "state"),
    ]:
        with pytest.raises(ValueError, match=f"^{name}"):
            call(**kw)
    t = u[..., 0].contiguous()
    with pytest.raises(ValueError, match="^state"):
        ssm.causal_conv_step(t, w, none[1], slots=_int([0]))
    with pytest.raises(ValueError, match="^x"):
        ssm.selective_step(t, t, A, B[..., 0].contiguous(), B[..., 0].contiguous(), none[0], slots=_int([0]))
