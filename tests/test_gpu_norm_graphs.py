"""Layer norm in captured graphs, in both orders of the tensors, and the gradients of wide groups
with the gate behind the norm."""
import numpy as np
import pytest

from tests.selective_cases import on_device
from tests.test_gpu_norm import DEV, _f32, _ssm, check, inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("order", ["tokens", "rows", "mixed"])
@pytest.mark.parametrize("gate,rms,H,L,groups", [("after", False, 96, 130, 3), ("before", True, 640, 70, 1), ("", False, 512, 257, 1),
                                                 ("after", False, 1200, 9, 1)])
def test_captured_training_step(order, gate, rms, H, L, groups):
    """Forward and backward captured once and replayed on new inputs, with the program's own eager work and
    synchronizations between the replays."""
    ssm = _ssm()
    a = inputs(21, "bf16", 2, H, L, gate)
    u, z, dy = (None if a[k] is None else on_device(a[k], "bf16", order) for k in ("u", "z", "dy"))
    more = dict(weight=_f32(a["weight"]), bias=_f32(a["bias"]), z=z, gate=gate or "after", rms=rms, groups=groups)

    def step():
        return dict(ssm.layer_norm(u, **more), **ssm.layer_norm_backward(u, dy, **more))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    gen = torch.Generator(device=DEV).manual_seed(22)
    for i in range(4):
        for t in (u, z, dy, more["weight"]):
            if t is not None:
                t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert (v is None) == (eager[k] is None) and (v is None or torch.equal(v, eager[k])), (i, k)


def test_two_captured_calls_on_one_workspace():
    """Graphs that share a workspace, replayed one after the other on a stream, each give what they gave alone."""
    ssm = _ssm()
    sets = []
    for seed, order, L in ((23, "tokens", 300), (24, "rows", 140)):
        a = inputs(seed, "f32", 2, 160, L, "before")
        u, z, dy = (on_device(a[k], "f32", order) for k in ("u", "z", "dy"))
        sets.append((u, dy, dict(weight=_f32(a["weight"]), bias=_f32(a["bias"]), z=z, gate="before")))
    ws = torch.full((1 << 23,), 255, dtype=torch.uint8, device=DEV)
    want = [ssm.layer_norm_backward(u, dy, **more) for u, dy, more in sets]
    torch.cuda.synchronize()
    graphs, got = [], []
    for u, dy, more in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(ssm.layer_norm_backward(u, dy, workspace=ws, **more))
    for _ in range(3):
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[i][k], want[i][k]) for i in range(2) for k in want[i])


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H", [5000, 9000, 16000])
@pytest.mark.parametrize("rms", [False, True])
def test_wide_groups_with_the_gate_behind(name, H, rms):
    """Groups of 512 threads, whose sums are in LDS above 8192 channels: the gate's gradient leaves before the second pass."""
    check(inputs(H, name, 1, H, 5, "after"), name, "tokens", 1, rms, "after")


def test_wide_groups_over_several_steps_of_a_workgroup():
    for H, L in ((5000, 600), (9000, 520)):
        check(inputs(H + 1, "bf16", 1, H, L, "after", shift=0.0), "bf16", "tokens", 1, False, "after")
