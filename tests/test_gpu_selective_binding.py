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
