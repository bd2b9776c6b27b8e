"""Host-side checks of the selective operators' C ABI (no GPU needed): struct
layouts agree with the header, sizes are what the layouts say, and bad
arguments are refused before anything reaches a device."""
import ctypes
import os
import subprocess

import pytest

ssm = pytest.importorskip("structured_state_space_amd.ssm", reason="HIP library not built")
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000000  # aligned dummy address: validation fails before any use
INVALID, WORKSPACE, UNSUPPORTED = ssm.ERR_INVALID_ARGUMENT, ssm.ERR_WORKSPACE, ssm.ERR_UNSUPPORTED
STRUCTS = {"ssm_view": ssm.View, "ssm_group_view": ssm.GroupView, "ssm_sequences": ssm.Sequences,
           "ssm_selective": ssm.Selective, "ssm_selective_grads": ssm.SelectiveGrads,
           "ssm_selective_token": ssm.SelectiveToken}


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
        want = getattr(STRUCTS[cls], field).offset if field else ctypes.sizeof(STRUCTS[cls])
        assert int(value) == want, name


def test_bytes():
    B = ssm.selective_bytes
    # states every 32 steps, a row of H x 16 floats each
    assert B(ssm.OP_SELECTIVE_SAVED, 2, 48, 16, 1, 33) == 2 * 2 * 48 * 16 * 4
    assert B(ssm.OP_SELECTIVE_SAVED, 2, 48, 40, 1, 33) == 2 * 2 * 48 * 64 * 4
    assert B(ssm.OP_SELECTIVE_SAVED, 1, 48, 16, 1, 33, 5, True) == (1 + 5) * 48 * 16 * 4
    # enough sequences and channels: no chunks, no workspace
    assert B(ssm.OP_SELECTIVE_SCAN, 16, 4096, 16, 1, 2048) == 0
    assert B(ssm.OP_SELECTIVE_SCAN, 1, 64, 16, 1, 4096) > 0
    assert B(ssm.OP_SELECTIVE_SCAN, 1, 64, 16, 1, 20) == 0
    assert B(ssm.OP_SELECTIVE_SCAN_BACKWARD, 2, 48, 16, 1, 33) >= 2 * 33 * 32 * 4 + 2 * 48 * 18 * 4
    assert B(ssm.OP_CAUSAL_CONV_BACKWARD, 2, 48, 4, 1, 33) >= 2 * 48 * 5 * 4


@pytest.mark.parametrize("args,code", [
    ((-1, 1, 8, 16, 1, 8, 1, 0), INVALID),
    ((4, 1, 8, 16, 1, 8, 1, 0), INVALID),
    ((0, 0, 8, 16, 1, 8, 0, 0), INVALID),
    ((0, 1, 0, 16, 1, 8, 1, 0), INVALID),
    ((0, 1, 8, 0, 1, 8, 1, 0), INVALID),
    ((0, 1, 8, 16, 3, 8, 1, 0), INVALID),       # groups that do not divide the channels
    ((0, 1, 8, 16, 0, 8, 1, 0), INVALID),
    ((0, 1, 8, 16, 1, 0, 1, 0), INVALID),
    ((0, 2, 8, 16, 1, 8, 3, 0), INVALID),       # sequences without offsets are the rows
    ((0, 2, 8, 16, 1, 8, 3, 1), INVALID),       # packed: one row
    ((0, 1, 8, 65, 1, 8, 1, 0), UNSUPPORTED),
    ((0, 1 << 20, 1 << 12, 16, 1, 8, 1 << 20, 0), UNSUPPORTED),
    ((0, 1, 8, 16, 1, 1 << 31, 1, 0), UNSUPPORTED),
    ((3, 1, 8, 0, 1, 8, 1, 0), INVALID),
    ((3, 1, 8, 5, 1, 8, 1, 0), UNSUPPORTED),
    ((0, 1 << 23, 64, 16, 1, 8, 1 << 23, 0), UNSUPPORTED),   # 2^32 threads in a launch
    ((2, 1 << 23, 64, 16, 1, 8, 1 << 23, 0), UNSUPPORTED),
    ((3, 1 << 24, 64, 4, 1, 8, 1 << 24, 0), UNSUPPORTED),
])
def test_bytes_rejects(args, code):
    out = ctypes.c_size_t(123)
    assert ssm.lib.ssm_selective_bytes(*args, ctypes.byref(out)) == code and out.value == 123
    assert ssm.lib.ssm_selective_bytes(0, 1, 8, 16, 1, 8, 1, 0, None) == INVALID


def _seq(**kw):
    return ssm.Sequences(**{**dict(Bsz=2, L=16, S=2), **kw})


def _view(**kw):
    return ssm.View(**{**dict(data=FAKE, sb=128, sh=16, sl=1), **kw})


BAD_SEQ = [
    (dict(Bsz=0), INVALID), (dict(L=0), INVALID), (dict(S=3), INVALID),
    (dict(offsets=FAKE), INVALID),                                  # two batch rows
    (dict(Bsz=1, S=2, offsets=FAKE, lengths=FAKE), INVALID),
    (dict(Bsz=1, S=2, offsets=FAKE + 2), INVALID),
    (dict(lengths=FAKE + 1), INVALID),
    (dict(slots=FAKE, n_slots=0), INVALID),
    (dict(slots=FAKE, n_slots=1 << 41), UNSUPPORTED),
    (dict(L=(1 << 31) - 8), UNSUPPORTED),
    (dict(Bsz=1 << 30, S=1 << 30), UNSUPPORTED),
]
BAD_VIEW = [
    (dict(data=None), INVALID), (dict(data=FAKE + 1), INVALID), (dict(sl=-1), INVALID), (dict(sh=-1), INVALID),
    (dict(sh=1 << 23), UNSUPPORTED), (dict(sl=1 << 23), UNSUPPORTED), (dict(sb=1 << 40), UNSUPPORTED),
]
BAD_OUT = BAD_VIEW + [(dict(sb=0), INVALID), (dict(sh=0), INVALID), (dict(sl=0), INVALID)]


def _conv(**kw):
    a = dict(dtype=ssm.BF16, seq=_seq(), H=8, W=4, u=_view(), w=FAKE, b=FAKE, s0=FAKE, s1=FAKE, y=_view())
    a.update(kw)
    return ssm.lib.ssm_causal_conv(a["dtype"], a["seq"], a["H"], a["W"], 1, a["u"], a["w"], a["b"], a["s0"], a["s1"],
                                   a["y"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(H=0), INVALID), (dict(W=0), INVALID),
    (dict(W=5), UNSUPPORTED), (dict(w=None), INVALID), (dict(w=FAKE + 2), INVALID), (dict(b=FAKE + 1), INVALID),
    (dict(s0=FAKE + 1), INVALID), (dict(s1=FAKE + 1), INVALID), (dict(W=1, s1=None), INVALID),
    (dict(W=1, s0=None), INVALID), (dict(seq=None), INVALID), (dict(u=None), INVALID), (dict(y=None), INVALID),
    (dict(dtype=ssm.F32, u=_view(data=FAKE + 2)), INVALID),
] + [(dict(seq=_seq(**k)), c) for k, c in BAD_SEQ] + [(dict(u=_view(**k)), c) for k, c in BAD_VIEW]
  + [(dict(y=_view(**k)), c) for k, c in BAD_OUT])
def test_conv_rejects(kw, code):
    assert _conv(**kw) == code


def _conv_back(**kw):
    a = dict(dtype=ssm.BF16, seq=_seq(), H=8, W=4, u=_view(), w=FAKE, b=FAKE, s0=FAKE, dy=_view(), ds1=FAKE,
             du=_view(), dw=FAKE, db=FAKE, ds0=FAKE, ws=FAKE, n=1 << 30)
    a.update(kw)
    return ssm.lib.ssm_causal_conv_backward(a["dtype"], a["seq"], a["H"], a["W"], 1, a["u"], a["w"], a["b"], a["s0"],
                                            a["dy"], a["ds1"], a["du"], a["dw"], a["db"], a["ds0"], a["ws"], a["n"],
                                            None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), INVALID), (dict(W=9), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(n=64), WORKSPACE),
    (dict(ws=FAKE + 64), INVALID), (dict(dw=FAKE + 1), INVALID), (dict(ds0=FAKE + 2), INVALID),
    (dict(W=1, s0=None, ds0=None), INVALID), (dict(seq=_seq(slots=FAKE, n_slots=4)), INVALID),
] + [(dict(seq=_seq(**k)), c) for k, c in BAD_SEQ if "slots" not in k]
  + [(dict(dy=_view(**k)), c) for k, c in BAD_VIEW] + [(dict(du=_view(**k)), c) for k, c in BAD_OUT])
def test_conv_backward_rejects(kw, code):
    assert _conv_back(**kw) == code


def _group(**kw):
    return ssm.GroupView(**{**dict(data=FAKE, sb=256, sg=256, sn=16, sl=1), **kw})


def _selective(**kw):
    base = dict(H=8, N=16, G=2, dtype=ssm.BF16, softplus=1, u=_view(), delta=_view(), z=_view(), B=_group(),
                C=_group(), A=FAKE, D=FAKE, delta_bias=FAKE, x_in=FAKE)
    return ssm.Selective(**{**base, **kw})


BAD_SELECTIVE = [
    (dict(dtype=3), INVALID), (dict(H=0), INVALID), (dict(N=0), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID),
    (dict(N=65), UNSUPPORTED), (dict(A=None), INVALID), (dict(A=FAKE + 2), INVALID), (dict(D=FAKE + 1), INVALID),
    (dict(delta_bias=FAKE + 2), INVALID), (dict(x_in=FAKE + 2), INVALID),
    (dict(B=_group(data=None)), INVALID), (dict(C=_group(sn=-1)), INVALID), (dict(C=_group(sn=1 << 23)), UNSUPPORTED),
    (dict(B=_group(sg=1 << 40)), UNSUPPORTED), (dict(B=_group(sl=1 << 23)), UNSUPPORTED),
] + [(dict(u=_view(**k)), c) for k, c in BAD_VIEW] + [(dict(delta=_view(**k)), c) for k, c in BAD_VIEW] \
  + [(dict(z=_view(**k)), c) for k, c in BAD_VIEW[1:]]


def _scan(**kw):
    a = dict(seq=_seq(), p=_selective(), y=_view(), x=FAKE, saved=None, sn=0, ws=FAKE, n=1 << 30)
    a.update(kw)
    return ssm.lib.ssm_selective_scan(a["seq"], a["p"], a["y"], a["x"], a["saved"], a["sn"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(seq=None), INVALID), (dict(p=None), INVALID), (dict(y=None, x=None), INVALID), (dict(x=FAKE + 2), INVALID),
    (dict(saved=FAKE, sn=16), WORKSPACE), (dict(saved=FAKE + 4, sn=1 << 30), INVALID),
    (dict(saved=FAKE, sn=1 << 30, seq=_seq(slots=FAKE, n_slots=4)), INVALID),
    (dict(ws=FAKE + 8), INVALID),
    (dict(seq=_seq(Bsz=1, S=1, L=4096), ws=None), WORKSPACE), (dict(seq=_seq(Bsz=1, S=1, L=4096), n=16), WORKSPACE),
] + [(dict(seq=_seq(**k)), c) for k, c in BAD_SEQ] + [(dict(p=_selective(**k)), c) for k, c in BAD_SELECTIVE]
  + [(dict(y=_view(**k)), c) for k, c in BAD_OUT if k != dict(data=None)])
def test_scan_rejects(kw, code):
    assert _scan(**kw) == code


def _grads(**kw):
    base = dict(du=_view(), ddelta=_view(), dz=_view(), dB=_group(), dC=_group(), dA=FAKE, dD=FAKE, ddelta_bias=FAKE,
                dx_in=FAKE)
    return ssm.SelectiveGrads(**{**base, **kw})


def _scan_back(**kw):
    a = dict(seq=_seq(), p=_selective(), saved=FAKE, sn=1 << 30, dy=_view(), dx=FAKE, g=_grads(), ws=FAKE, n=1 << 30)
    a.update(kw)
    return ssm.lib.ssm_selective_scan_backward(a["seq"], a["p"], a["saved"], a["sn"], a["dy"], a["dx"], a["g"],
                                               a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(saved=None), INVALID), (dict(sn=16), WORKSPACE), (dict(saved=FAKE + 16), INVALID), (dict(ws=None), WORKSPACE),
    (dict(n=128), WORKSPACE), (dict(ws=FAKE + 4), INVALID), (dict(g=None), INVALID), (dict(dx=FAKE + 1), INVALID),
    (dict(g=_grads(dA=None)), INVALID), (dict(g=_grads(dD=FAKE + 1)), INVALID), (dict(g=_grads(dz=_view(data=None))), INVALID),
    (dict(p=_selective(z=_view(data=None))), INVALID),      # dz without z
    (dict(g=_grads(dB=_group(sn=0))), INVALID), (dict(g=_grads(dC=_group(sl=0))), INVALID),
    (dict(g=_grads(dC=_group(sg=0))), INVALID), (dict(g=_grads(dB=_group(data=None))), INVALID),
    (dict(seq=_seq(slots=FAKE, n_slots=4)), INVALID),
] + [(dict(seq=_seq(**k)), c) for k, c in BAD_SEQ if "slots" not in k]
  + [(dict(p=_selective(**k)), c) for k, c in BAD_SELECTIVE] + [(dict(dy=_view(**k)), c) for k, c in BAD_VIEW]
  + [(dict(g=_grads(du=_view(**k))), c) for k, c in BAD_OUT]
  + [(dict(g=_grads(ddelta=_view(**k))), c) for k, c in BAD_OUT])
def test_scan_backward_rejects(kw, code):
    assert _scan_back(**kw) == code


def _token(**kw):
    base = dict(Bsz=2, H=8, N=16, G=2, dtype=ssm.F16, softplus=1, slots=None, n_slots=2, u=FAKE, delta=FAKE, z=FAKE,
                B=FAKE, C=FAKE, y=FAKE, u_stride=8, delta_stride=8, z_stride=8, y_stride=8, B_stride=32, B_group=16,
                B_state=1, C_stride=32, C_group=16, C_state=1, A=FAKE, D=FAKE, delta_bias=FAKE, x=FAKE)
    return ssm.lib.ssm_selective_step(ssm.SelectiveToken(**{**base, **kw}), None)


@pytest.mark.parametrize("kw,code", [
    (dict(Bsz=0), INVALID), (dict(H=0), INVALID), (dict(N=0), INVALID), (dict(G=5), INVALID), (dict(dtype=4), INVALID),
    (dict(N=65), UNSUPPORTED), (dict(Bsz=1 << 30), UNSUPPORTED), (dict(Bsz=1 << 24), UNSUPPORTED), (dict(u=None), INVALID), (dict(x=None), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(x=FAKE + 2), INVALID), (dict(slots=FAKE, n_slots=0), INVALID),
    (dict(slots=FAKE + 2), INVALID), (dict(u_stride=-1), INVALID), (dict(B_state=-1), INVALID), (dict(C_state=1 << 32), UNSUPPORTED), (dict(y_stride=0), INVALID),
    (dict(B_stride=1 << 32), UNSUPPORTED), (dict(slots=FAKE, n_slots=1 << 40), UNSUPPORTED),
])
def test_step_rejects(kw, code):
    assert _token(**kw) == code
    assert ssm.lib.ssm_selective_step(None, None) == INVALID


def _conv_step(**kw):
    a = dict(dtype=ssm.F32, Bsz=2, H=8, W=4, u=FAKE, us=8, w=FAKE, b=FAKE, state=FAKE, slots=None, n=2, y=FAKE, ys=8)
    a.update(kw)
    return ssm.lib.ssm_causal_conv_step(a["dtype"], a["Bsz"], a["H"], a["W"], 1, a["u"], a["us"], a["w"], a["b"],
                                        a["state"], a["slots"], a["n"], a["y"], a["ys"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), INVALID), (dict(Bsz=0), INVALID), (dict(W=0), INVALID), (dict(W=5), UNSUPPORTED),
    (dict(state=None), INVALID), (dict(W=1), INVALID), (dict(u=None), INVALID), (dict(y=FAKE + 2), INVALID),
    (dict(us=-1), INVALID), (dict(ys=0), INVALID), (dict(us=1 << 32), UNSUPPORTED), (dict(slots=FAKE, n=0), INVALID),
    (dict(slots=FAKE + 1), INVALID), (dict(H=1 << 31), UNSUPPORTED),
])
def test_conv_step_rejects(kw, code):
    assert _conv_step(**kw) == code


def test_binding_refuses_host_tensors_and_wrong_shapes():
    u = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        ssm.causal_conv(u, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        ssm.selective_scan(u, u, torch.zeros(4, 16), torch.zeros(1, 1, 16, 8), torch.zeros(1, 1, 16, 8))
    with pytest.raises(ValueError):
        ssm.selective_step(u[..., 0], u[..., 0], torch.zeros(4, 16), torch.zeros(1, 1, 16), torch.zeros(1, 1, 16), None)
    with pytest.raises(ValueError):
        ssm.causal_conv_step(u, torch.zeros(4, 4), None)


def test_packed_calls_are_split_by_the_same_rule():
    B = ssm.selective_bytes
    for op in (ssm.OP_SELECTIVE_SCAN, ssm.OP_SELECTIVE_SCAN_BACKWARD):
        size = lambda H, S, packed, N=16: B(op, 1, H, N, 1, 4096, S, packed)  # noqa: E731
        parts = lambda H, S: 4096 * (H // 64) * 32 * 4 + (S + 1) * H * 18 * 4  # noqa: E731  of the backward pass
        whole = lambda H, S: 0 if op == ssm.OP_SELECTIVE_SCAN else parts(H, S)  # noqa: E731
        # 64 channels a workgroup: three chunks of 10240 are worth it, two of 12288 are not
        for H in (10240, 8192):
            assert size(H, 2, True) > whole(H, 2) and size(H, 1, False) > whole(H, 0)
        for H in (12288, 16384):
            assert size(H, 2, True) == whole(H, 2) and size(H, 1, False) == whole(H, 0)
