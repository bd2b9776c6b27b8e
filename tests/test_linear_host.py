"""Host-side checks of the linear attention and layer norm C ABI (no GPU needed):
struct layouts agree with the header, sizes are what the layouts say, and bad
arguments are refused before anything reaches a device."""
import ctypes
import os
import subprocess

import pytest

ssm = pytest.importorskip("structured_state_space_amd.ssm", reason="HIP library not built")
torch = pytest.importorskip("torch")

from tests.test_selective_host import BAD_OUT, BAD_SEQ, BAD_VIEW, FAKE, INVALID, UNSUPPORTED, WORKSPACE, _seq, _view  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"ssm_linear": ssm.Linear, "ssm_linear_grads": ssm.LinearGrads, "ssm_linear_token": ssm.LinearToken,
           "ssm_norm": ssm.Norm}
BF16, F32 = torch.bfloat16, torch.float32


def test_struct_layouts_match_the_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ssm.h"', "int main(void) {"]
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, *_ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, value = line.split()
        cls, _, field = name.partition(".")
        assert int(value) == (getattr(STRUCTS[cls], field).offset if field else ctypes.sizeof(STRUCTS[cls])), name


def test_bytes():
    B = ssm.linear_bytes
    saved, fwd, bwd = ssm.OP_LINEAR_SAVED, ssm.OP_LINEAR_ATTENTION, ssm.OP_LINEAR_ATTENTION_BACKWARD
    # states every 64 steps (float32: 32), keys padded to 16, values to 32
    assert B(saved, BF16, 2, 4, 20, 40, 2, 65) == 2 * 2 * 4 * 32 * 64 * 4
    assert B(saved, F32, 2, 4, 20, 40, 2, 65) == 2 * 3 * 4 * 32 * 64 * 4
    assert B(saved, BF16, 1, 4, 64, 64, 2, 65, 5, True) == (1 + 5) * 4 * 64 * 64 * 4
    # enough heads: no segments, no workspace; a long row of few heads has them
    assert B(fwd, BF16, 4, 64, 128, 64, 1, 2048) == 0
    assert B(fwd, BF16, 1, 2, 128, 64, 1, 4096) > 0
    assert B(fwd, BF16, 1, 2, 128, 64, 1, 64) == 0
    assert B(bwd, BF16, 2, 4, 64, 64, 2, 65) >= B(saved, BF16, 2, 4, 64, 64, 2, 65)


@pytest.mark.parametrize("args,code", [
    ((-1, 1, 1, 8, 16, 16, 1, 8, 1, 0), INVALID), ((3, 1, 1, 8, 16, 16, 1, 8, 1, 0), INVALID),
    ((0, 3, 1, 8, 16, 16, 1, 8, 1, 0), INVALID), ((0, 1, 0, 8, 16, 16, 1, 8, 0, 0), INVALID),
    ((0, 1, 1, 0, 16, 16, 1, 8, 1, 0), INVALID), ((0, 1, 1, 8, 0, 16, 1, 8, 1, 0), INVALID),
    ((0, 1, 1, 8, 16, 0, 1, 8, 1, 0), INVALID), ((0, 1, 1, 8, 16, 16, 3, 8, 1, 0), INVALID),
    ((0, 1, 1, 8, 16, 16, 0, 8, 1, 0), INVALID), ((0, 1, 1, 8, 16, 16, 1, 0, 1, 0), INVALID),
    ((0, 1, 2, 8, 16, 16, 1, 8, 3, 0), INVALID), ((0, 1, 2, 8, 16, 16, 1, 8, 3, 1), INVALID),
    ((0, 1, 1, 8, 257, 16, 1, 8, 1, 0), UNSUPPORTED), ((0, 1, 1, 8, 16, 257, 1, 8, 1, 0), UNSUPPORTED),
    ((0, 1, 1 << 20, 1 << 12, 16, 16, 1, 8, 1 << 20, 0), UNSUPPORTED),
    ((0, 1, 1, 8, 16, 16, 1, 1 << 31, 1, 0), UNSUPPORTED),
    ((0, 1, 1 << 23, 1, 16, 16, 1, 8, 1 << 23, 0), UNSUPPORTED),      # 2^32 threads in a launch
])
def test_bytes_rejects(args, code):
    out = ctypes.c_size_t(123)
    assert ssm.lib.ssm_linear_bytes(*args, ctypes.byref(out)) == code and out.value == 123
    assert ssm.lib.ssm_linear_bytes(0, 1, 1, 8, 16, 16, 1, 8, 1, 0, None) == INVALID


def _group(**kw):
    return ssm.GroupView(**{**dict(data=FAKE, sb=4096, sg=256, sn=16, sl=1), **kw})


BAD_GROUP = [(dict(data=None), INVALID), (dict(data=FAKE + 1), INVALID), (dict(sl=-1), INVALID), (dict(sn=-1), INVALID),
             (dict(sg=-1), INVALID), (dict(sn=1 << 23), UNSUPPORTED), (dict(sl=1 << 23), UNSUPPORTED),
             (dict(sg=1 << 40), UNSUPPORTED), (dict(sb=1 << 40), UNSUPPORTED)]
BAD_GROUP_OUT = BAD_GROUP + [(dict(sb=0), INVALID), (dict(sg=0), INVALID), (dict(sn=0), INVALID), (dict(sl=0), INVALID)]


def _linear(**kw):
    return ssm.Linear(**{**dict(H=4, G=2, N=16, P=16, dtype=ssm.BF16, scale=1.0, q=_group(), k=_group(), v=_group(),
                                g=_view(), beta=_view(), D=FAKE, x_in=FAKE), **kw})


def _forward(seq=None, y=_group(), x_out=FAKE, saved=FAKE, size=1 << 40, ws=FAKE, n=1 << 40, null=None, **kw):
    p = None if null == "p" else _linear(**kw)
    return ssm.lib.ssm_linear_attention(None if null == "seq" else seq or _seq(), p, y, x_out, saved, size, ws, n, None)


BAD_LINEAR = [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(H=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
    (dict(N=0), INVALID), (dict(P=0), INVALID), (dict(N=257), UNSUPPORTED), (dict(P=257), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(D=FAKE + 2), INVALID),
    (dict(x_in=FAKE + 1), INVALID), (dict(g=_view(data=None)), INVALID), (dict(g=_view(data=FAKE + 2)), INVALID),
    (dict(beta=_view(sl=-1)), INVALID), (dict(beta=_view(sl=1 << 23)), UNSUPPORTED), (dict(null="p"), INVALID),
    (dict(null="seq"), INVALID),
] + [({n: _group(**k)}, c) for n in ("q", "k", "v") for k, c in BAD_GROUP]


@pytest.mark.parametrize("kw,code", BAD_LINEAR + [
    (dict(y=_group(**k)), c) for k, c in BAD_GROUP_OUT if k != dict(data=None)] + [
    (dict(x_out=FAKE + 2), INVALID), (dict(saved=FAKE + 64), INVALID), (dict(ws=FAKE + 64), INVALID),
    (dict(size=100), WORKSPACE), (dict(y=None, x_out=None, saved=None), INVALID),
    (dict(y=_group(data=None), x_out=None, saved=None), INVALID),
    (dict(seq=_seq(slots=FAKE, n_slots=4)), INVALID),                            # states are not saved with slots
    (dict(seq=_seq(Bsz=1, S=1, L=8192), ws=None), WORKSPACE), (dict(seq=_seq(Bsz=1, S=1, L=8192), n=100), WORKSPACE),
] + [(dict(seq=_seq(**k), saved=None), c) for k, c in BAD_SEQ])
def test_forward_rejects(kw, code):
    assert _forward(**kw) == code


def _grads(**kw):
    return ssm.LinearGrads(**{**dict(dq=_group(), dk=_group(), dv=_group(), dg=_view(), dbeta=_view(), dD=FAKE, dx_in=FAKE), **kw})


def _backward(seq=None, saved=FAKE, size=1 << 40, dy=_group(), dx=FAKE, ws=FAKE, n=1 << 40, grads=None, null=None, **kw):
    p = None if null == "p" else _linear(**kw)
    g = None if null == "grads" else _grads(**(grads or {}))
    return ssm.lib.ssm_linear_attention_backward(None if null == "seq" else seq or _seq(), p, saved, size, dy, dx, g, ws, n, None)


@pytest.mark.parametrize("kw,code", BAD_LINEAR + [
    (dict(null="grads"), INVALID), (dict(saved=None), INVALID), (dict(saved=FAKE + 64), INVALID), (dict(size=100), WORKSPACE),
    (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE), (dict(ws=FAKE + 8), INVALID), (dict(dx=FAKE + 2), INVALID),
    (dict(dy=None), INVALID), (dict(seq=_seq(slots=FAKE, n_slots=4)), INVALID),
    (dict(beta=_view(data=None)), INVALID), (dict(D=None), INVALID),             # gradients of what was not given
    (dict(grads=dict(dD=FAKE + 1)), INVALID), (dict(grads=dict(dx_in=FAKE + 1)), INVALID),
] + [(dict(dy=_group(**k)), c) for k, c in BAD_GROUP]
  + [(dict(grads={n: _group(**k)}), c) for n in ("dq", "dk", "dv") for k, c in BAD_GROUP_OUT]
  + [(dict(grads=dict(dg=_view(**{"data": FAKE, **k}))), c) for k, c in BAD_OUT]
  + [(dict(grads=dict(dbeta=_view(**k))), c) for k, c in BAD_OUT if k != dict(data=None)]
  + [(dict(seq=_seq(**k)), INVALID if "slots" in k else c) for k, c in BAD_SEQ])
def test_backward_rejects(kw, code):
    assert _backward(**kw) == code


def _token(**kw):
    strides = {f"{n}_{k}": 64 for n, ks in (("q", ("stride", "group", "key")), ("k", ("stride", "group", "key")),
                                          ("v", ("stride", "head", "value")), ("y", ("stride", "head", "value")),
                                          ("g", ("stride", "head")), ("beta", ("stride", "head"))) for k in ks}
    base = dict(Bsz=2, H=4, G=2, N=16, P=16, dtype=ssm.F16, scale=1.0, slots=None, n_slots=2, q=FAKE, k=FAKE, v=FAKE, y=FAKE,
                g=FAKE, beta=FAKE, D=FAKE, x=FAKE, **strides)
    return ssm.lib.ssm_linear_attention_step(ssm.LinearToken(**{**base, **kw}), None)


@pytest.mark.parametrize("kw,code", [
    (dict(Bsz=0), INVALID), (dict(H=0), INVALID), (dict(G=3), INVALID), (dict(N=0), INVALID), (dict(P=0), INVALID),
    (dict(dtype=4), INVALID), (dict(N=257), UNSUPPORTED), (dict(P=257), UNSUPPORTED), (dict(Bsz=1 << 30), UNSUPPORTED),
    (dict(Bsz=1 << 24), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(g=None), INVALID), (dict(y=None), INVALID), (dict(x=None), INVALID), (dict(q=FAKE + 1), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(g=FAKE + 2), INVALID), (dict(x=FAKE + 2), INVALID), (dict(slots=FAKE, n_slots=0), INVALID),
    (dict(slots=FAKE + 2), INVALID), (dict(scale=float("inf")), INVALID), (dict(q_key=-1), INVALID), (dict(beta_head=-1), INVALID),
    (dict(y_stride=0), INVALID), (dict(y_head=0), INVALID), (dict(y_value=0), INVALID), (dict(v_head=1 << 32), UNSUPPORTED),
    (dict(slots=FAKE, n_slots=1 << 40), UNSUPPORTED),
])
def test_step_rejects(kw, code):
    assert _token(**kw) == code
    assert ssm.lib.ssm_linear_attention_step(None, None) == INVALID


# -------------------------------------------------------------- layer norm ----

def _norm(**kw):
    return ssm.Norm(**{**dict(Bsz=2, H=8, L=16, G=2, dtype=ssm.BF16, rms=0, gate=1, eps=1e-5, u=_view(), z=_view(), weight=FAKE,
                              bias=FAKE), **kw})


BAD_NORM = [
    (dict(Bsz=0), INVALID), (dict(H=0), INVALID), (dict(L=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
    (dict(dtype=3), INVALID), (dict(gate=3), INVALID), (dict(gate=-1), INVALID), (dict(gate=0), INVALID),   # z without a gate
    (dict(z=_view(data=None)), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(weight=FAKE + 2), INVALID), (dict(bias=FAKE + 1), INVALID),
    (dict(Bsz=1 << 30), UNSUPPORTED), (dict(L=1 << 31), UNSUPPORTED),
] + [({n: _view(**k)}, c) for n in ("u", "z") for k, c in BAD_VIEW]


@pytest.mark.parametrize("kw,code", BAD_NORM + [(dict(y=_view(**k)), c) for k, c in BAD_OUT] + [(dict(y=None), INVALID)])
def test_norm_rejects(kw, code):
    y = kw.get("y", _view())
    assert ssm.lib.ssm_layer_norm(_norm(**{k: v for k, v in kw.items() if k != "y"}), y, None) == code
    assert ssm.lib.ssm_layer_norm(None, _view(), None) == INVALID


@pytest.mark.parametrize("kw,code", BAD_NORM + [(dict(dy=_view(**k)), c) for k, c in BAD_VIEW] + [
    ({n: _view(**k)}, c) for n in ("du", "dz") for k, c in BAD_OUT] + [
    (dict(ws=None), WORKSPACE), (dict(n=8), WORKSPACE), (dict(ws=FAKE + 8), INVALID), (dict(dw=FAKE + 2), INVALID),
    (dict(db=FAKE + 1), INVALID)])
def test_norm_backward_rejects(kw, code):
    a = dict(dy=_view(), du=_view(), dz=_view(), dw=FAKE, db=FAKE, ws=FAKE, n=1 << 40)
    a.update({k: v for k, v in kw.items() if k in a})
    p = _norm(**{k: v for k, v in kw.items() if k not in a})
    assert ssm.lib.ssm_layer_norm_backward(p, a["dy"], a["du"], a["dz"], a["dw"], a["db"], a["ws"], a["n"], None) == code


def test_norm_bytes():
    out = ctypes.c_size_t()
    assert ssm.lib.ssm_layer_norm_bytes(2, 8, 16, 3, ctypes.byref(out)) == INVALID
    assert ssm.lib.ssm_layer_norm_bytes(2, 8, 16, 2, None) == INVALID
    assert ssm.lib.ssm_layer_norm_bytes(2, 8, 16, 2, ctypes.byref(out)) == ssm.OK and out.value >= 2 * 8 * 4


@pytest.mark.parametrize("sizes", [(65536, 8192, 1, 64), (32768, 8192, 1, 128), (1 << 19, 512, 1, 8), (16, 8192, 4096, 64)])
def test_norms_of_many_tokens_have_a_workspace(sizes):
    """More than 2^22 (token, group) rows: what the order of contiguous channels takes is not refused by the other's grid."""
    out = ctypes.c_size_t()
    assert ssm.lib.ssm_layer_norm_bytes(*sizes, ctypes.byref(out)) == ssm.OK and out.value > 0


def test_norms_are_refused_by_the_grid_of_their_own_order():
    """Forwards, every second channel of 2^22 rows, and contiguous ones of 2^32 threads (refused before anything runs)."""
    for kw in (dict(Bsz=32768, H=8192, L=1, G=128, u=_view(sb=16384, sh=2)), dict(Bsz=1 << 20, H=512, L=1, G=512, u=_view(sh=1))):
        p = _norm(**{**dict(gate=0, z=_view(data=None)), **kw})
        assert ssm.lib.ssm_layer_norm(p, _view(sb=8192, sh=1), None) == UNSUPPORTED
    out = ctypes.c_size_t()
    assert ssm.lib.ssm_layer_norm_bytes(1, 1 << 24, 1, 1 << 24, ctypes.byref(out)) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q, v, g = torch.zeros(1, 1, 4, 8), torch.zeros(1, 2, 4, 8), torch.zeros(1, 2, 8)
    for call in (lambda: ssm.linear_attention(q, q, v, g), lambda: ssm.linear_attention_backward(q, q, v, g, v),
                 lambda: ssm.linear_attention_step(q[..., 0], q[..., 0], v[..., 0], g[..., 0], None),
                 lambda: ssm.layer_norm(v[0]), lambda: ssm.layer_norm_backward(v[0], v[0]),
                 lambda: ssm.layer_norm(v[0], gate="inside")):
        with pytest.raises(ValueError):
            call()
