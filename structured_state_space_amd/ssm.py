"""Python binding of the C ABI in include/ssm.h (argument marshalling only).

Every step of the filter path runs in the HIP library; this module only checks
tensor shapes and dtypes, allocates workspaces with torch, and passes device
pointers plus torch's current HIP stream.  Importing it loads the in-tree
library built by structured_state_space_amd/build.py and raises ImportError
when it is missing: there is no CPU fallback.

torch is imported first so that the library binds to the HIP runtime torch has
already loaded (both use the libamdhip64.so.7 soname).
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libssm_hip.so")

# return codes and statuses, as declared in include/ssm.h
OK = 0
ERR_INVALID_ARGUMENT = 1
ERR_WORKSPACE = 2
ERR_DEVICE = 3
ERR_UNSUPPORTED = 4
ERR_SCRATCH_LIMIT = 5
NOALLOC_SCRATCH_BYTES = 64 << 20
ST_OK = 0
ST_RESONANT_CORRECTION = 16
ST_RESONANT_DIAGONAL = 17
ST_SINGULAR_BILINEAR = 18
ST_INVALID_STEP = 19
ST_UNPREPARED = 20
OP_DISCRETIZE, OP_KERNEL_GEN, OP_FFTCONV, OP_FORWARD, OP_FORWARD_COMPLEX, OP_HIPPO = 0, 1, 2, 3, 4, 5
OP_STEP_PREPARED = 6
HIPPO_LEGS, HIPPO_LEGT, HIPPO_LAGT = 0, 1, 2
HIPPO_KINDS = {"legs": HIPPO_LEGS, "legt": HIPPO_LEGT, "lagt": HIPPO_LAGT}

EXPORTS = ("ssm_workspace_bytes", "ssm_transform_lengths", "ssm_forward_form", "ssm_status_string",
           "ssm_discretize", "ssm_kernel_gen", "ssm_fftconv", "ssm_forward", "ssm_forward_profiled", "ssm_step",
           "ssm_forward_complex", "ssm_hippo_dplr", "ssm_step_prepare", "ssm_step_prepared",
           "ssm_forward_noalloc", "ssm_selective_bytes", "ssm_causal_conv", "ssm_causal_conv_backward",
           "ssm_causal_conv_step", "ssm_selective_scan", "ssm_selective_scan_backward", "ssm_selective_step",
           "ssm_linear_bytes", "ssm_linear_attention", "ssm_linear_attention_backward", "ssm_linear_attention_step",
           "ssm_layer_norm_bytes", "ssm_layer_norm", "ssm_layer_norm_backward")

# element types and operation ids of the selective operators
F32, BF16, F16 = 0, 1, 2
OP_SELECTIVE_SCAN, OP_SELECTIVE_SCAN_BACKWARD, OP_SELECTIVE_SAVED, OP_CAUSAL_CONV_BACKWARD = 0, 1, 2, 3
OP_LINEAR_ATTENTION, OP_LINEAR_ATTENTION_BACKWARD, OP_LINEAR_SAVED = 0, 1, 2
GATES = {"none": 0, "before": 1, "after": 2}
_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


class View(ctypes.Structure):
    """ssm_view"""
    _fields_ = [("data", ctypes.c_void_p)] + [(k, ctypes.c_int64) for k in ("sb", "sh", "sl")]


class GroupView(ctypes.Structure):
    """ssm_group_view"""
    _fields_ = [("data", ctypes.c_void_p)] + [(k, ctypes.c_int64) for k in ("sb", "sg", "sn", "sl")]


class Sequences(ctypes.Structure):
    """ssm_sequences"""
    _fields_ = ([(k, ctypes.c_int64) for k in ("Bsz", "L", "S")]
                + [(k, ctypes.c_void_p) for k in ("offsets", "lengths", "slots")] + [("n_slots", ctypes.c_int64)])


class Selective(ctypes.Structure):
    """ssm_selective"""
    _fields_ = ([(k, ctypes.c_int64) for k in ("H", "N", "G")] + [(k, ctypes.c_int32) for k in ("dtype", "softplus")]
                + [(k, View) for k in ("u", "delta", "z")] + [(k, GroupView) for k in ("B", "C")]
                + [(k, ctypes.c_void_p) for k in ("A", "D", "delta_bias", "x_in")])


class SelectiveGrads(ctypes.Structure):
    """ssm_selective_grads"""
    _fields_ = ([(k, View) for k in ("du", "ddelta", "dz")] + [(k, GroupView) for k in ("dB", "dC")]
                + [(k, ctypes.c_void_p) for k in ("dA", "dD", "ddelta_bias", "dx_in")])


class SelectiveToken(ctypes.Structure):
    """ssm_selective_token"""
    _fields_ = ([(k, ctypes.c_int64) for k in ("Bsz", "H", "N", "G")]
                + [(k, ctypes.c_int32) for k in ("dtype", "softplus")]
                + [("slots", ctypes.c_void_p), ("n_slots", ctypes.c_int64)]
                + [(k, ctypes.c_void_p) for k in ("u", "delta", "z", "B", "C", "y")]
                + [(k, ctypes.c_int64) for k in ("u_stride", "delta_stride", "z_stride", "y_stride", "B_stride",
                                                 "B_group", "B_state", "C_stride", "C_group", "C_state")]
                + [(k, ctypes.c_void_p) for k in ("A", "D", "delta_bias", "x")])


class Linear(ctypes.Structure):
    """ssm_linear"""
    _fields_ = ([(k, ctypes.c_int64) for k in ("H", "G", "N", "P")]
                + [("dtype", ctypes.c_int32), ("scale", ctypes.c_float)] + [(k, GroupView) for k in ("q", "k", "v")]
                + [(k, View) for k in ("g", "beta")] + [(k, ctypes.c_void_p) for k in ("D", "x_in")])


class LinearGrads(ctypes.Structure):
    """ssm_linear_grads"""
    _fields_ = ([(k, GroupView) for k in ("dq", "dk", "dv")] + [(k, View) for k in ("dg", "dbeta")]
                + [(k, ctypes.c_void_p) for k in ("dD", "dx_in")])


class LinearToken(ctypes.Structure):
    """ssm_linear_token"""
    _fields_ = ([(k, ctypes.c_int64) for k in ("Bsz", "H", "G", "N", "P")]
                + [("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]
                + [("slots", ctypes.c_void_p), ("n_slots", ctypes.c_int64)]
                + [(k, ctypes.c_void_p) for k in ("q", "k", "v", "y", "g", "beta")]
                + [(k, ctypes.c_int64) for k in ("q_stride", "q_group", "q_key", "k_stride", "k_group", "k_key",
                                                 "v_stride", "v_head", "v_value", "y_stride", "y_head", "y_value",
                                                 "g_stride", "g_head", "beta_stride", "beta_head")]
                + [(k, ctypes.c_void_p) for k in ("D", "x")])


class Norm(ctypes.Structure):
    """ssm_norm"""
    _fields_ = ([(k, ctypes.c_int64) for k in ("Bsz", "H", "L", "G")]
                + [(k, ctypes.c_int32) for k in ("dtype", "rms", "gate")] + [("eps", ctypes.c_float)]
                + [(k, View) for k in ("u", "z")] + [(k, ctypes.c_void_p) for k in ("weight", "bias")])


class SSMError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {status_string(code)} (code {code})")
        self.code = code


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"HIP library not built: {_LIB_PATH} is missing "
                          "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
    lib = ctypes.CDLL(_LIB_PATH)
    i64, vp, sz, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.ssm_workspace_bytes.argtypes = [i32, i64, i64, i64, i64, i64, ctypes.POINTER(sz)]
    lib.ssm_workspace_bytes.restype = i32
    lib.ssm_transform_lengths.argtypes = [i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.ssm_transform_lengths.restype = i32
    lib.ssm_forward_form.argtypes = [i64, i64, i64, ctypes.POINTER(ctypes.c_int32)]
    lib.ssm_forward_form.restype = i32
    lib.ssm_status_string.argtypes = [i32]
    lib.ssm_status_string.restype = ctypes.c_char_p
    lib.ssm_discretize.argtypes = [i64, i64, i64, i64] + [vp] * 10 + [vp, sz, vp]
    lib.ssm_discretize.restype = i32
    lib.ssm_kernel_gen.argtypes = [i64, i64, i64, i64] + [vp] * 9 + [vp, sz, vp]
    lib.ssm_kernel_gen.restype = i32
    lib.ssm_fftconv.argtypes = [i64, i64, i64, vp, i64, vp, vp, vp, vp, sz, vp]
    lib.ssm_fftconv.restype = i32
    lib.ssm_forward.argtypes = [i64, i64, i64, i64, i64] + [vp] * 11 + [vp, sz, vp]
    lib.ssm_forward.restype = i32
    lib.ssm_forward_profiled.argtypes = [i64, i64, i64, i64, i64] + [vp] * 11 + [vp, sz, vp, vp, ctypes.c_int32]
    lib.ssm_forward_profiled.restype = i32
    lib.ssm_step.argtypes = [i64, i64, i64, i64, i64] + [vp] * 11 + [ctypes.c_int32, vp]
    lib.ssm_step.restype = i32
    lib.ssm_step_prepare.argtypes = [i64, i64, i64] + [vp] * 7 + [sz, vp, vp]
    lib.ssm_step_prepare.restype = i32
    lib.ssm_step_prepared.argtypes = [i64, i64, i64, i64, i64, vp, sz] + [vp] * 5 + [ctypes.c_int32, vp]
    lib.ssm_step_prepared.restype = i32
    lib.ssm_forward_complex.argtypes = [i64, i64, i64, i64, i64] + [vp] * 12 + [vp, sz, vp]
    lib.ssm_forward_complex.restype = i32
    lib.ssm_forward_noalloc.argtypes = [i64, i64, i64, i64, i64] + [vp] * 11 + [vp]
    lib.ssm_forward_noalloc.restype = i32
    lib.ssm_hippo_dplr.argtypes = [i32, i64, ctypes.c_double, i64, vp, i64, vp] + [vp] * 5 + [vp, sz, vp]
    lib.ssm_hippo_dplr.restype = i32
    view, seqs = ctypes.POINTER(View), ctypes.POINTER(Sequences)
    lib.ssm_selective_bytes.argtypes = [i32, i64, i64, i64, i64, i64, i64, i32, ctypes.POINTER(sz)]
    lib.ssm_selective_bytes.restype = i32
    lib.ssm_causal_conv.argtypes = [i32, seqs, i64, i64, i32, view, vp, vp, vp, vp, view, vp]
    lib.ssm_causal_conv.restype = i32
    lib.ssm_causal_conv_backward.argtypes = ([i32, seqs, i64, i64, i32, view, vp, vp, vp, view, vp, view]
                                             + [vp] * 4 + [sz, vp])
    lib.ssm_causal_conv_backward.restype = i32
    lib.ssm_causal_conv_step.argtypes = [i32, i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp]
    lib.ssm_causal_conv_step.restype = i32
    lib.ssm_selective_scan.argtypes = [seqs, ctypes.POINTER(Selective), view, vp, vp, sz, vp, sz, vp]
    lib.ssm_selective_scan.restype = i32
    lib.ssm_selective_scan_backward.argtypes = [seqs, ctypes.POINTER(Selective), vp, sz, view, vp,
                                                ctypes.POINTER(SelectiveGrads), vp, sz, vp]
    lib.ssm_selective_scan_backward.restype = i32
    lib.ssm_selective_step.argtypes = [ctypes.POINTER(SelectiveToken), vp]
    lib.ssm_selective_step.restype = i32
    group, linear = ctypes.POINTER(GroupView), ctypes.POINTER(Linear)
    lib.ssm_linear_bytes.argtypes = [i32, i32] + [i64] * 7 + [i32, ctypes.POINTER(sz)]
    lib.ssm_linear_bytes.restype = i32
    lib.ssm_linear_attention.argtypes = [seqs, linear, group, vp, vp, sz, vp, sz, vp]
    lib.ssm_linear_attention.restype = i32
    lib.ssm_linear_attention_backward.argtypes = [seqs, linear, vp, sz, group, vp, ctypes.POINTER(LinearGrads), vp, sz, vp]
    lib.ssm_linear_attention_backward.restype = i32
    lib.ssm_linear_attention_step.argtypes = [ctypes.POINTER(LinearToken), vp]
    lib.ssm_linear_attention_step.restype = i32
    norm = ctypes.POINTER(Norm)
    lib.ssm_layer_norm_bytes.argtypes = [i64] * 4 + [ctypes.POINTER(sz)]
    lib.ssm_layer_norm_bytes.restype = i32
    lib.ssm_layer_norm.argtypes = [norm, view, vp]
    lib.ssm_layer_norm.restype = i32
    lib.ssm_layer_norm_backward.argtypes = [norm, view, view, view, vp, vp, vp, sz, vp]
    lib.ssm_layer_norm_backward.restype = i32
    return lib


lib = _load()


def status_string(code: int) -> str:
    return lib.ssm_status_string(int(code)).decode()


def transform_lengths(L: int):
    M, n = ctypes.c_int64(), ctypes.c_int64()
    rc = lib.ssm_transform_lengths(int(L), ctypes.byref(M), ctypes.byref(n))
    if rc != OK:
        raise SSMError("ssm_transform_lengths", rc)
    return M.value, n.value


def forward_form(Bsz: int, H: int, L: int) -> int:
    """ssm_forward_form: 1 (single launch), 2 (root values + convolution with
    spectra) or 3 (root values, spectra, convolution)."""
    out = ctypes.c_int32()
    rc = lib.ssm_forward_form(int(Bsz), int(H), int(L), ctypes.byref(out))
    if rc != OK:
        raise SSMError("ssm_forward_form", rc)
    return out.value


def workspace_bytes(op: int, Bsz: int, H: int, N: int, r: int, L: int) -> int:
    out = ctypes.c_size_t()
    rc = lib.ssm_workspace_bytes(int(op), int(Bsz), int(H), int(N), int(r), int(L), ctypes.byref(out))
    if rc != OK:
        raise SSMError("ssm_workspace_bytes", rc)
    return out.value


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(t, name, dtype, shape, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != tuple(shape):
        got = (None if not isinstance(t, torch.Tensor) else (t.dtype, tuple(t.shape)))
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {got}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name}: must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _params(Lambda, P, Q, B, Cv, dt):
    H, N = Lambda.shape
    r = P.shape[2]
    dev = Lambda.device
    _check(Lambda, "Lambda", torch.complex64, (H, N), dev)
    _check(P, "P", torch.complex64, (H, N, r), dev)
    _check(Q, "Q", torch.complex64, (H, N, r), dev)
    _check(B, "B", torch.complex64, (H, N), dev)
    _check(Cv, "C", torch.complex64, (H, N), dev)
    _check(dt, "dt", torch.float32, (H,), dev)
    return H, N, r, dev


def _workspace(nbytes, device, workspace=None):
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def discretize(Lambda, P, Q, B, C, dt, L, want_bbar=True, want_abar=False, want_ctilde=True):
    """ssm_discretize: returns dict(Bbar, Abar, Ctilde, status) (None where not asked)."""
    H, N, r, dev = _params(Lambda, P, Q, B, C, dt)
    Bbar = torch.empty((H, N), dtype=torch.complex64, device=dev) if want_bbar else None
    Abar = torch.empty((H, N, N), dtype=torch.complex64, device=dev) if want_abar else None
    Ct = torch.empty((H, N), dtype=torch.complex64, device=dev) if want_ctilde else None
    status = torch.empty((H,), dtype=torch.int32, device=dev)
    rc = lib.ssm_discretize(H, N, r, int(L), _ptr(Lambda), _ptr(P), _ptr(Q), _ptr(B), _ptr(C), _ptr(dt),
                            _ptr(Bbar), _ptr(Abar), _ptr(Ct), _ptr(status), None, 0, _stream(dev))
    if rc != OK:
        raise SSMError("ssm_discretize", rc)
    return dict(Bbar=Bbar, Abar=Abar, Ctilde=Ct, status=status)


def kernel_gen(Lambda, P, Q, B, Ctilde, dt, L, want_kernel=True, want_roots=False, workspace=None):
    """ssm_kernel_gen: returns dict(K [H,L] c64, roots [H,M] c64, status [H] i32)."""
    H, N, r, dev = _params(Lambda, P, Q, B, Ctilde, dt)
    M, _ = transform_lengths(L)
    K = torch.empty((H, L), dtype=torch.complex64, device=dev) if want_kernel else None
    roots = torch.empty((H, M), dtype=torch.complex64, device=dev) if want_roots else None
    status = torch.empty((H,), dtype=torch.int32, device=dev)
    nbytes = workspace_bytes(OP_KERNEL_GEN, 1, H, N, r, L)
    ws = _workspace(nbytes, dev, workspace)
    rc = lib.ssm_kernel_gen(H, N, r, int(L), _ptr(Lambda), _ptr(P), _ptr(Q), _ptr(B), _ptr(Ctilde), _ptr(dt),
                            _ptr(K), _ptr(roots), _ptr(status), _ptr(ws), nbytes, _stream(dev))
    if rc != OK:
        raise SSMError("ssm_kernel_gen", rc)
    return dict(K=K, roots=roots, status=status)


def fftconv(K, u, D=None, y=None, workspace=None):
    """ssm_fftconv: y = K * u + D u.  K: float32 [H,L] or complex64 [H,L] (real part used)."""
    Bsz, H, L = u.shape
    dev = u.device
    _check(u, "u", torch.float32, (Bsz, H, L), dev)
    if K.dtype == torch.complex64:
        _check(K, "K", torch.complex64, (H, L), dev)
        stride = 2
    else:
        _check(K, "K", torch.float32, (H, L), dev)
        stride = 1
    _check(D, "D", torch.float32, (H,), dev)
    if y is None:
        y = torch.empty_like(u)
    _check(y, "y", torch.float32, (Bsz, H, L), dev)
    nbytes = workspace_bytes(OP_FFTCONV, Bsz, H, 1, 1, L)
    ws = _workspace(nbytes, dev, workspace)
    rc = lib.ssm_fftconv(Bsz, H, L, _ptr(K), stride, _ptr(D), _ptr(u), _ptr(y), _ptr(ws), nbytes, _stream(dev))
    if rc != OK:
        raise SSMError("ssm_fftconv", rc)
    return y


def forward(Lambda, P, Q, B, Ctilde, dt, D, u, want_kernel=False, y=None, K_out=None, status=None,
            workspace=None, events=None, repeat=1):
    """ssm_forward: returns dict(y [Bsz,H,L] f32, K [H,L] c64 or None, status [H] i32).

    events: optional four torch.cuda.Event(enable_timing=True); then the call goes
    through ssm_forward_profiled, which launches each of its three stages
    `repeat` times and records the events around them."""
    H, N, r, dev = _params(Lambda, P, Q, B, Ctilde, dt)
    Bsz, H2, L = u.shape
    if H2 != H:
        raise ValueError("u: channel count does not match the parameters")
    _check(u, "u", torch.float32, (Bsz, H, L), dev)
    _check(D, "D", torch.float32, (H,), dev)
    if y is None:
        y = torch.empty_like(u)
    _check(y, "y", torch.float32, (Bsz, H, L), dev)
    if K_out is None and want_kernel:
        K_out = torch.empty((H, L), dtype=torch.complex64, device=dev)
    _check(K_out, "K_out", torch.complex64, (H, L), dev)
    if status is None:
        status = torch.empty((H,), dtype=torch.int32, device=dev)
    _check(status, "status", torch.int32, (H,), dev)
    nbytes = workspace_bytes(OP_FORWARD, Bsz, H, N, r, L)
    ws = _workspace(nbytes, dev, workspace)
    args = (Bsz, H, N, r, L, _ptr(Lambda), _ptr(P), _ptr(Q), _ptr(B), _ptr(Ctilde), _ptr(dt), _ptr(D), _ptr(u),
            _ptr(y), _ptr(K_out), _ptr(status), _ptr(ws), nbytes, _stream(dev))
    if events is None:
        rc = lib.ssm_forward(*args)
        name = "ssm_forward"
    else:
        # torch creates its events lazily; record once so each has a handle
        for e in events:
            if e.cuda_event == 0:
                e.record()
        arr = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
        rc = lib.ssm_forward_profiled(*args, arr, int(repeat))
        name = "ssm_forward_profiled"
    if rc != OK:
        raise SSMError(name, rc)
    return dict(y=y, K=K_out, status=status)


def forward_noalloc(Lambda, P, Q, B, Ctilde, dt, D, u, y=None, K_out=None, status=None):
    """ssm_forward_noalloc: ssm_forward with the library's fixed per-GPU scratch
    instead of a workspace (the call allocates nothing when y, K_out and status
    are given).  Returns dict(y, K, status) as forward does."""
    H, N, r, dev = _params(Lambda, P, Q, B, Ctilde, dt)
    Bsz, H2, L = u.shape
    if H2 != H:
        raise ValueError("u: channel count does not match the parameters")
    _check(u, "u", torch.float32, (Bsz, H, L), dev)
    _check(D, "D", torch.float32, (H,), dev)
    if y is None:
        y = torch.empty_like(u)
    _check(y, "y", torch.float32, (Bsz, H, L), dev)
    _check(K_out, "K_out", torch.complex64, (H, L), dev)
    if status is None:
        status = torch.empty((H,), dtype=torch.int32, device=dev)
    _check(status, "status", torch.int32, (H,), dev)
    rc = lib.ssm_forward_noalloc(Bsz, H, N, r, L, _ptr(Lambda), _ptr(P), _ptr(Q), _ptr(B), _ptr(Ctilde), _ptr(dt),
                                 _ptr(D), _ptr(u), _ptr(y), _ptr(K_out), _ptr(status), _stream(dev))
    if rc != OK:
        raise SSMError("ssm_forward_noalloc", rc)
    return dict(y=y, K=K_out, status=status)


def forward_complex(Lambda, P, Q, B, Ctilde, dt, D, u, want_kernel=False, workspace=None):
    """ssm_forward_complex: returns dict(y_re, y_im [Bsz,H,L] f32 (the real and
    imaginary parts of y), K [H,L] c64 or None, status [H] i32)."""
    H, N, r, dev = _params(Lambda, P, Q, B, Ctilde, dt)
    Bsz, H2, L = u.shape
    if H2 != H:
        raise ValueError("u: channel count does not match the parameters")
    _check(u, "u", torch.float32, (Bsz, H, L), dev)
    _check(D, "D", torch.float32, (H,), dev)
    y_re, y_im = torch.empty_like(u), torch.empty_like(u)
    K_out = torch.empty((H, L), dtype=torch.complex64, device=dev) if want_kernel else None
    status = torch.empty((H,), dtype=torch.int32, device=dev)
    nbytes = workspace_bytes(OP_FORWARD_COMPLEX, Bsz, H, N, r, L)
    ws = _workspace(nbytes, dev, workspace)
    rc = lib.ssm_forward_complex(Bsz, H, N, r, L, _ptr(Lambda), _ptr(P), _ptr(Q), _ptr(B), _ptr(Ctilde), _ptr(dt),
                                 _ptr(D), _ptr(u), _ptr(y_re), _ptr(y_im), _ptr(K_out), _ptr(status), _ptr(ws),
                                 nbytes, _stream(dev))
    if rc != OK:
        raise SSMError("ssm_forward_complex", rc)
    return dict(y_re=y_re, y_im=y_im, K=K_out, status=status)


def step(Lambda, P, Q, B, C, dt, D, u, x=None, y=None, status=None, lanes=0):
    """ssm_step: T steps of the recurrence from the state x (zeros when None);
    returns dict(y [Bsz,H,T] f32, x [Bsz,H,N] c64 (the state after the last
    step, updated in place when given), status [H] i32).  lanes: 64 (one
    sequence per wave), 16 (N <= 64: four per wave) or 0 (chosen per call)."""
    H, N, r, dev = _params(Lambda, P, Q, B, C, dt)
    Bsz, H2, T = u.shape
    if H2 != H:
        raise ValueError("u: channel count does not match the parameters")
    _check(u, "u", torch.float32, (Bsz, H, T), dev)
    _check(D, "D", torch.float32, (H,), dev)
    if x is None:
        x = torch.zeros((Bsz, H, N), dtype=torch.complex64, device=dev)
    _check(x, "x", torch.complex64, (Bsz, H, N), dev)
    if y is None:
        y = torch.empty_like(u)
    _check(y, "y", torch.float32, (Bsz, H, T), dev)
    if status is None:
        status = torch.empty((H,), dtype=torch.int32, device=dev)
    _check(status, "status", torch.int32, (H,), dev)
    rc = lib.ssm_step(Bsz, H, N, r, T, _ptr(Lambda), _ptr(P), _ptr(Q), _ptr(B), _ptr(C), _ptr(dt), _ptr(D), _ptr(u),
                      _ptr(y), _ptr(x), _ptr(status), int(lanes), _stream(dev))
    if rc != OK:
        raise SSMError("ssm_step", rc)
    return dict(y=y, x=x, status=status)


def step_prepare(Lambda, P, Q, B, C, dt, prep=None, status=None):
    """ssm_step_prepare: the per-channel set-up of the step mode, once per
    parameter set.  Returns dict(prep (uint8 device buffer of the float32
    constants), status [H] i32, H, N, r), which step_prepared takes."""
    H, N, r, dev = _params(Lambda, P, Q, B, C, dt)
    nbytes = workspace_bytes(OP_STEP_PREPARED, 0, H, N, r, 0)
    if prep is None:
        prep = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif not (isinstance(prep, torch.Tensor) and prep.dtype == torch.uint8 and prep.is_cuda and prep.device == dev
              and prep.is_contiguous() and prep.numel() >= nbytes):
        raise ValueError(f"prep: expected a contiguous uint8 tensor of at least {nbytes} bytes on {dev}")
    if status is None:
        status = torch.empty((H,), dtype=torch.int32, device=dev)
    _check(status, "status", torch.int32, (H,), dev)
    rc = lib.ssm_step_prepare(H, N, r, _ptr(Lambda), _ptr(P), _ptr(Q), _ptr(B), _ptr(C), _ptr(dt), _ptr(prep),
                              prep.numel(), _ptr(status), _stream(dev))
    if rc != OK:
        raise SSMError("ssm_step_prepare", rc)
    return dict(prep=prep, status=status, H=H, N=N, r=r)


def step_prepared(prepared, D, u, x=None, y=None, status=None, lanes=0):
    """ssm_step_prepared: T steps of the recurrence from the state x (zeros
    when None) with the constants of step_prepare's result `prepared`;
    returns dict(y, x, status) as step does, bit for bit in the same layout.
    lanes: 64, 16 (N <= 64) or 0 (chosen by the library per call)."""
    prep, H, N, r = prepared["prep"], prepared["H"], prepared["N"], prepared["r"]
    dev = prep.device
    Bsz, H2, T = u.shape
    if H2 != H:
        raise ValueError("u: channel count does not match the prepared constants")
    _check(u, "u", torch.float32, (Bsz, H, T), dev)
    _check(D, "D", torch.float32, (H,), dev)
    if x is None:
        x = torch.zeros((Bsz, H, N), dtype=torch.complex64, device=dev)
    _check(x, "x", torch.complex64, (Bsz, H, N), dev)
    if y is None:
        y = torch.empty_like(u)
    _check(y, "y", torch.float32, (Bsz, H, T), dev)
    if status is None:
        status = torch.empty((H,), dtype=torch.int32, device=dev)
    _check(status, "status", torch.int32, (H,), dev)
    rc = lib.ssm_step_prepared(Bsz, H, N, r, T, _ptr(prep), prep.numel(), _ptr(D), _ptr(u), _ptr(y), _ptr(x),
                               _ptr(status), int(lanes), _stream(dev))
    if rc != OK:
        raise SSMError("ssm_step_prepared", rc)
    return dict(y=y, x=x, status=status)


def hippo_dplr(kind, N, theta=1.0, B=None, C=None, want_v=False, device="cuda:0", workspace=None):
    """ssm_hippo_dplr: DPLR parameters of a HiPPO generator.  kind is "legs",
    "legt" or "lagt" (or its SSM_HIPPO_* code); B [nb,N] and C [nc,N] are
    complex64 device tensors or None.  Returns dict(Lambda [N], P [N,rank],
    V [N,N] or None, Bt [nb,N] or None, Ct [nc,N] or None), all complex64."""
    code = HIPPO_KINDS[kind] if isinstance(kind, str) else int(kind)
    dev = torch.device(device)
    if B is not None:
        dev = B.device
        _check(B, "B", torch.complex64, (B.shape[0], N), dev)
    if C is not None:
        dev = C.device if B is None else dev
        _check(C, "C", torch.complex64, (C.shape[0], N), dev)
    rank = 2 if code == HIPPO_LEGT else 1
    Lam = torch.empty((N,), dtype=torch.complex64, device=dev)
    P = torch.empty((N, rank), dtype=torch.complex64, device=dev)
    V = torch.empty((N, N), dtype=torch.complex64, device=dev) if want_v else None
    nb = 0 if B is None else B.shape[0]
    nc = 0 if C is None else C.shape[0]
    Bt = torch.empty_like(B) if B is not None else None
    Ct = torch.empty_like(C) if C is not None else None
    nbytes = workspace_bytes(OP_HIPPO, 0, 0, N, 0, 0)
    ws = _workspace(nbytes, dev, workspace)
    rc = lib.ssm_hippo_dplr(code, N, float(theta), nb, _ptr(B), nc, _ptr(C), _ptr(Lam), _ptr(P), _ptr(V), _ptr(Bt),
                            _ptr(Ct), _ptr(ws), nbytes, _stream(dev))
    if rc != OK:
        raise SSMError("ssm_hippo_dplr", rc)
    return dict(Lambda=Lam, P=P, V=V, Bt=Bt, Ct=Ct)


# ---- selective operators ----
#
# Activations are float32, bfloat16 or float16 tensors [Bsz, H, L] (B and C
# [Bsz, G, N, L]) with any strides: a projection's [Bsz, L, H] output goes in as
# its .transpose(1, 2), a slice as it is.  Outputs that the call makes are
# dense, in the order of the input they belong to.
#
# As everywhere in this binding, autograd does not see the calls: outputs never
# require gradients, also where inputs do.  The gradients are the *_backward
# calls, for use in a torch.autograd.Function or by hand.
#
# Where no sequence runs (steps that offsets or lengths leave out, rows whose slot
# names no state) a y that is given stays as it was, and one that the call makes
# holds what its memory held: give y=torch.zeros_like(u) where such places are read.
# Gradients that a call makes are zero there.


def _address(t):
    return None if t is None else t.data_ptr()


def _queue(device):
    # the current stream's handle, without the Stream object around it (1.9 us)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _strides(t):
    # a dimension of one element has no stride
    return [s if n > 1 else 0 for s, n in zip(t.stride(), t.shape)] if 1 in t.shape else t.stride()


def _scratch(nbytes, device, workspace):
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    return _workspace(nbytes, device, workspace)


def _view(t):
    return View() if t is None else View(t.data_ptr(), *_strides(t))


def _group_view(t):
    return GroupView(t.data_ptr(), *_strides(t))


def _activation(t, name, dtype, shape, device):
    # shape: a tuple
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape:
        got = (None if not isinstance(t, torch.Tensor) else (t.dtype, tuple(t.shape)))
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {got}")
    if t.device != device:
        raise ValueError(f"{name}: must be on {device}")


def _first(u, dims):
    if not isinstance(u, torch.Tensor) or u.dim() != dims or u.dtype not in _TYPES or not u.is_cuda:
        raise ValueError(f"u: expected a float32, bfloat16 or float16 device tensor of {dims} dimensions")
    if u.numel() == 0:
        raise ValueError("u: has no elements")
    return u.device, _TYPES[u.dtype]


def _like(t, empty=True):
    """A dense output for t [Bsz,...,L], with the steps stored last where t's are
    contiguous and first (behind the batch) elsewhere."""
    if t.stride(-1) == 1:
        out = torch.empty(t.shape, dtype=t.dtype, device=t.device)
    elif t.dim() == 3:
        Bsz, H, L = t.shape
        out = torch.empty_strided((Bsz, H, L), (H * L, 1, H), dtype=t.dtype, device=t.device)
    else:
        Bsz, G, N, L = t.shape
        out = torch.empty_strided((Bsz, G, N, L), (G * N * L, N, 1, G * N), dtype=t.dtype, device=t.device)
    return out if empty else out.zero_()


class _on:
    """The device of a call's tensors, made current where it is not."""

    def __init__(self, device):
        self.switch = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.switch is not None:
            self.switch.__enter__()

    def __exit__(self, *exc):
        if self.switch is not None:
            self.switch.__exit__(*exc)


def _count(Bsz, offsets):
    """The number of sequences."""
    if offsets is None:
        return Bsz
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets: expected torch.int32 [S+1]")
    return offsets.shape[0] - 1


def _sequences(Bsz, L, device, offsets, lengths, slots, n_slots):
    """(ssm_sequences, the tensors it points to are the caller's)"""
    S = _count(Bsz, offsets)
    if offsets is not None:
        if lengths is not None:
            raise ValueError("offsets and lengths: give one of them")
        if Bsz != 1:
            raise ValueError("offsets: need one batch row")
        _check(offsets, "offsets", torch.int32, (S + 1,), device)
    _check(lengths, "lengths", torch.int32, (S,), device)
    _check(slots, "slots", torch.int32, (S,), device)
    ptr = [None if t is None else t.data_ptr() for t in (offsets, lengths, slots)]
    return Sequences(Bsz, L, S, *ptr, 0 if slots is None else n_slots)


def _states(t, name, dtype, S, slots, tail, device):
    """Rows of a state array: S of them, or any number of them with slots."""
    if t is None:
        return 0
    rows = S if slots is None or not isinstance(t, torch.Tensor) or t.dim() < 1 else t.shape[0]
    _check(t, name, dtype, (rows, *tail), device)
    if rows == 0:
        raise ValueError(f"{name}: has no rows")
    return rows


def _pool(a, b, names):
    if a and b and a != b:
        raise ValueError(f"{names}: must have the same number of rows")
    return a or b


def _any_slot(H):
    # no state array: a slot only says whether its sequence runs, and any row that a
    # pool of H channels can have does (the library takes pools up to 2^40 / H rows)
    return min(2 ** 31, 2 ** 40 // H)


def selective_bytes(op, Bsz, H, N, G, L, S=None, packed=False):
    """ssm_selective_bytes"""
    out = ctypes.c_size_t()
    rc = lib.ssm_selective_bytes(int(op), int(Bsz), int(H), int(N), int(G), int(L), int(Bsz if S is None else S),
                                 int(bool(packed)), ctypes.byref(out))
    if rc != OK:
        raise SSMError("ssm_selective_bytes", rc)
    return out.value


def causal_conv(u, weight, bias=None, silu=False, state=None, state_out=None, want_state=False, offsets=None,
                lengths=None, slots=None, y=None):
    """ssm_causal_conv: y_t = act(bias + sum_k weight[:, k] u_{t-W+1+k}) over u
    [Bsz,H,L], weight float32 [H,W], bias [H].  state: the W - 1 inputs before
    the first step, [S,H,W-1] of u's type (with slots, a pool [rows,H,W-1]).
    The inputs before the next step go to state_out (which may be state), or to
    a new tensor with want_state.  offsets, lengths, slots as in the header
    (slots without states: a negative one skips its sequence).  y is not written
    where no sequence runs, and not seen by autograd.  Returns dict(y, state)."""
    dev, code = _first(u, 3)
    Bsz, H, L = u.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight: expected torch.float32 [H, W]")
    W = weight.shape[1]
    _check(weight, "weight", torch.float32, (H, W), dev)
    _check(bias, "bias", torch.float32, (H,), dev)
    S = _count(Bsz, offsets)
    tail = (H, W - 1)
    if W == 1 and (state is not None or state_out is not None):
        raise ValueError("state: a convolution of width 1 has none")
    rows = _pool(_states(state, "state", u.dtype, S, slots, tail, dev),
                 _states(state_out, "state_out", u.dtype, S, slots, tail, dev), "state and state_out")
    with _on(dev):
        if state_out is None and want_state and W > 1:
            if slots is not None:
                raise ValueError("want_state: with slots give state_out")
            state_out = torch.empty((S, *tail), dtype=u.dtype, device=dev)
        seq = _sequences(Bsz, L, dev, offsets, lengths, slots, rows or _any_slot(H))
        if y is None:
            y = _like(u)
        else:
            _activation(y, "y", u.dtype, (Bsz, H, L), dev)
        rc = lib.ssm_causal_conv(code, seq, H, W, int(silu), _view(u), _address(weight), _address(bias), _address(state),
                                 _address(state_out), _view(y), _queue(dev))
    if rc != OK:
        raise SSMError("ssm_causal_conv", rc)
    return dict(y=y, state=state_out)


def causal_conv_backward(u, weight, dy, bias=None, silu=False, state=None, dstate=None, want_dstate=False,
                         offsets=None, lengths=None, workspace=None):
    """ssm_causal_conv_backward: gradients for dy [Bsz,H,L] of y and dstate
    (float32 [S,H,W-1], or None) of the final state; the other arguments as in
    the forward call.  Returns dict(du, dweight, dbias (None without bias),
    dstate (of the initial state, with want_dstate))."""
    dev, code = _first(u, 3)
    Bsz, H, L = u.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight: expected torch.float32 [H, W]")
    W = weight.shape[1]
    _check(weight, "weight", torch.float32, (H, W), dev)
    _check(bias, "bias", torch.float32, (H,), dev)
    _activation(dy, "dy", u.dtype, (Bsz, H, L), dev)
    if W == 1 and (state is not None or dstate is not None):
        raise ValueError("state: a convolution of width 1 has none")
    with _on(dev):
        seq = _sequences(Bsz, L, dev, offsets, lengths, None, 0)
        tail = (seq.S, H, W - 1)
        _check(state, "state", u.dtype, tail, dev)
        _check(dstate, "dstate", torch.float32, tail, dev)
        du = _like(u, offsets is None and lengths is None)
        f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)  # noqa: E731
        dweight, dbias = f32(H, W), f32(H) if bias is not None else None
        dstate_in = f32(*tail) if want_dstate and W > 1 else None
        nbytes = selective_bytes(OP_CAUSAL_CONV_BACKWARD, Bsz, H, W, 1, L, seq.S, offsets is not None)
        ws = _scratch(nbytes, dev, workspace)
        rc = lib.ssm_causal_conv_backward(code, seq, H, W, int(silu), _view(u), _address(weight), _address(bias),
                                          _address(state), _view(dy), _address(dstate), _view(du), _address(dweight),
                                          _address(dbias), _address(dstate_in), _address(ws), nbytes, _queue(dev))
    if rc != OK:
        raise SSMError("ssm_causal_conv_backward", rc)
    return dict(du=du, dweight=dweight, dbias=dbias, dstate=dstate_in)


def causal_conv_step(u, weight, state, bias=None, silu=False, slots=None, y=None):
    """ssm_causal_conv_step: the convolution of one token per sequence, u [Bsz,H]
    (rows any number of elements apart); state [Bsz,H,W-1] (with slots, a pool
    [rows,H,W-1]) moves on in place.  y's rows whose slot names no state are not
    written.  Returns dict(y, state)."""
    dev, code = _first(u, 2)
    Bsz, H = u.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight: expected torch.float32 [H, W]")
    W = weight.shape[1]
    _check(weight, "weight", torch.float32, (H, W), dev)
    _check(bias, "bias", torch.float32, (H,), dev)
    _check(slots, "slots", torch.int32, (Bsz,), dev)
    if (state is None) != (W == 1):
        raise ValueError("state: needed for every width but 1")
    rows = _states(state, "state", u.dtype, Bsz, slots, (H, W - 1), dev)
    u_row = _row_stride(u, "u")
    with _on(dev):
        if y is None:
            y = torch.empty_like(u, memory_format=torch.contiguous_format)
        else:
            _activation(y, "y", u.dtype, (Bsz, H), dev)
        rc = lib.ssm_causal_conv_step(code, Bsz, H, W, int(silu), u.data_ptr(), u_row, weight.data_ptr(),
                                      _address(bias), _address(state), _address(slots), rows or _any_slot(H), y.data_ptr(),
                                      _row_stride(y, "y"), _queue(dev))
    if rc != OK:
        raise SSMError("ssm_causal_conv_step", rc)
    return dict(y=y, state=state)


def _row_stride(t, name):
    strides, shape = t.stride(), t.shape
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return strides[0] if shape[0] > 1 else 0


def _selective(u, delta, A, B, C, D, z, delta_bias, softplus, x0):
    dev, code = _first(u, 3)
    Bsz, H, L = u.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A: expected torch.float32 [H, N]")
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        raise ValueError("B: expected [Bsz, G, N, L]")
    N, G = A.shape[1], B.shape[1]
    _activation(delta, "delta", u.dtype, (Bsz, H, L), dev)
    _activation(B, "B", u.dtype, (Bsz, G, N, L), dev)
    _activation(C, "C", u.dtype, (Bsz, G, N, L), dev)
    if z is not None:
        _activation(z, "z", u.dtype, (Bsz, H, L), dev)
    _check(A, "A", torch.float32, (H, N), dev)
    _check(D, "D", torch.float32, (H,), dev)
    _check(delta_bias, "delta_bias", torch.float32, (H,), dev)
    if x0 is not None and not isinstance(x0, torch.Tensor):
        raise ValueError("x0: expected a torch.float32 tensor")
    args = Selective(H, N, G, code, int(softplus), _view(u), _view(delta), _view(z), _group_view(B), _group_view(C),
                     *(None if t is None else t.data_ptr() for t in (A, D, delta_bias, x0)))
    return dev, Bsz, H, L, N, G, args


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False, x0=None, x_out=None,
                   want_state=False, save=False, offsets=None, lengths=None, slots=None, y=None, workspace=None):
    """ssm_selective_scan: x_t = exp(dt_t A) x_{t-1} + dt_t u_t B_t,
    y_t = (C_t . x_t + D u_t) silu(z_t), dt = softplus(delta + delta_bias), over
    u, delta, z [Bsz,H,L], B, C [Bsz,G,N,L], A float32 [H,N], D, delta_bias
    float32 [H].  x0: the states before the first step, float32 [S,H,N] (with
    slots, a pool [rows,H,N]); the states after the last go to x_out (which may
    be x0), or to a new tensor with want_state.  save keeps what
    selective_scan_backward needs.  offsets, lengths, slots as in the header
    (slots without states: a negative one skips its sequence).  y is not written
    where no sequence runs, and not seen by autograd.  Returns dict(y, x, saved)."""
    dev, Bsz, H, L, N, G, args = _selective(u, delta, A, B, C, D, z, delta_bias, softplus, x0)
    S = _count(Bsz, offsets)
    rows = _pool(_states(x0, "x0", torch.float32, S, slots, (H, N), dev),
                 _states(x_out, "x_out", torch.float32, S, slots, (H, N), dev), "x0 and x_out")
    if slots is not None and (save or (want_state and x_out is None)):
        raise ValueError("slots: give x_out, and no save")
    with _on(dev):
        if x_out is None and want_state:
            x_out = torch.empty((S, H, N), dtype=torch.float32, device=dev)
        seq = _sequences(Bsz, L, dev, offsets, lengths, slots, rows or _any_slot(H))
        if y is None:
            y = _like(u)
        else:
            _activation(y, "y", u.dtype, (Bsz, H, L), dev)
        nbytes = selective_bytes(OP_SELECTIVE_SCAN, Bsz, H, N, G, L, S, offsets is not None)
        ws = _scratch(nbytes, dev, workspace) if nbytes else None
        saved, sbytes = None, 0
        if save:
            sbytes = selective_bytes(OP_SELECTIVE_SAVED, Bsz, H, N, G, L, S, offsets is not None)
            saved = torch.empty(sbytes, dtype=torch.uint8, device=dev)
        rc = lib.ssm_selective_scan(seq, args, _view(y), _address(x_out), _address(saved), sbytes, _address(ws), nbytes,
                                    _queue(dev))
    if rc != OK:
        raise SSMError("ssm_selective_scan", rc)
    return dict(y=y, x=x_out, saved=saved)


def selective_scan_backward(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, softplus=False, x0=None,
                            dx=None, saved=None, offsets=None, lengths=None, workspace=None):
    """ssm_selective_scan_backward: gradients for dy [Bsz,H,L] of y and dx
    (float32 [S,H,N], or None) of the final states; the other arguments as in the
    forward call, saved from it (None: the states are computed again).  Returns
    dict(du, ddelta, dA, dB, dC, dD, dz, ddelta_bias, dx0), None for the
    gradient of what was not given."""
    dev, Bsz, H, L, N, G, args = _selective(u, delta, A, B, C, D, z, delta_bias, softplus, x0)
    _activation(dy, "dy", u.dtype, (Bsz, H, L), dev)
    with _on(dev):
        seq = _sequences(Bsz, L, dev, offsets, lengths, None, 0)
        S, packed = seq.S, offsets is not None
        _check(x0, "x0", torch.float32, (S, H, N), dev)
        _check(dx, "dx", torch.float32, (S, H, N), dev)
        sbytes = selective_bytes(OP_SELECTIVE_SAVED, Bsz, H, N, G, L, S, packed)
        if saved is None:
            saved = torch.empty(sbytes, dtype=torch.uint8, device=dev)
            nbytes = selective_bytes(OP_SELECTIVE_SCAN, Bsz, H, N, G, L, S, packed)
            ws = _scratch(nbytes, dev, None) if nbytes else None
            rc = lib.ssm_selective_scan(seq, args, None, None, _address(saved), sbytes, _address(ws), nbytes, _queue(dev))
            if rc != OK:
                raise SSMError("ssm_selective_scan", rc)
        elif not (isinstance(saved, torch.Tensor) and saved.dtype == torch.uint8 and saved.device == dev
                  and saved.is_contiguous()):
            raise ValueError(f"saved: expected the uint8 tensor of the forward call on {dev}")
        whole = offsets is None and lengths is None
        f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)  # noqa: E731
        du, ddelta, dz = _like(u, whole), _like(delta, whole), _like(z, whole) if z is not None else None
        dB, dC, dA = _like(B, whole), _like(C, whole), f32(H, N)
        dD, dbias = f32(H) if D is not None else None, f32(H) if delta_bias is not None else None
        dx0 = f32(S, H, N) if x0 is not None else None
        grads = SelectiveGrads(_view(du), _view(ddelta), _view(dz), _group_view(dB), _group_view(dC),
                               *(None if t is None else t.data_ptr() for t in (dA, dD, dbias, dx0)))
        nbytes = selective_bytes(OP_SELECTIVE_SCAN_BACKWARD, Bsz, H, N, G, L, S, packed)
        ws = _scratch(nbytes, dev, workspace)
        rc = lib.ssm_selective_scan_backward(seq, args, _address(saved), saved.numel(), _view(dy), _address(dx), grads,
                                             _address(ws), nbytes, _queue(dev))
    if rc != OK:
        raise SSMError("ssm_selective_scan_backward", rc)
    return dict(du=du, ddelta=ddelta, dA=dA, dB=dB, dC=dC, dD=dD, dz=dz, ddelta_bias=dbias, dx0=dx0)


def selective_step(u, delta, A, B, C, x, D=None, z=None, delta_bias=None, softplus=False, slots=None, y=None):
    """ssm_selective_step: the scan of one token per sequence, u, delta, z
    [Bsz,H] (rows any number of elements apart), B, C [Bsz,G,N] (any strides); x float32
    [Bsz,H,N] (with slots, a pool [rows,H,N]) moves on in place.  y's rows whose
    slot names no state are not written.  Returns dict(y, x)."""
    dev, code = _first(u, 2)
    Bsz, H = u.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A: expected torch.float32 [H, N]")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B: expected [Bsz, G, N]")
    N, G = A.shape[1], B.shape[1]
    _activation(delta, "delta", u.dtype, (Bsz, H), dev)
    _activation(B, "B", u.dtype, (Bsz, G, N), dev)
    _activation(C, "C", u.dtype, (Bsz, G, N), dev)
    if z is not None:
        _activation(z, "z", u.dtype, (Bsz, H), dev)
    _check(A, "A", torch.float32, (H, N), dev)
    _check(D, "D", torch.float32, (H,), dev)
    _check(delta_bias, "delta_bias", torch.float32, (H,), dev)
    _check(slots, "slots", torch.int32, (Bsz,), dev)
    if x is None:
        raise ValueError("x: needed")
    rows = _states(x, "x", torch.float32, Bsz, slots, (H, N), dev)
    u_row, delta_row, z_row = _row_stride(u, "u"), _row_stride(delta, "delta"), 0 if z is None else _row_stride(z, "z")
    B_strides, C_strides = _strides(B), _strides(C)
    with _on(dev):
        if y is None:
            y = torch.empty_like(u, memory_format=torch.contiguous_format)
        else:
            _activation(y, "y", u.dtype, (Bsz, H), dev)
        args = SelectiveToken(Bsz, H, N, G, code, int(softplus), _address(slots), rows, u.data_ptr(),
                              delta.data_ptr(), _address(z), B.data_ptr(), C.data_ptr(), y.data_ptr(), u_row,
                              delta_row, z_row, _row_stride(y, "y"), *B_strides, *C_strides, A.data_ptr(),
                              _address(D), _address(delta_bias), x.data_ptr())
        rc = lib.ssm_selective_step(args, _queue(dev))
    if rc != OK:
        raise SSMError("ssm_selective_step", rc)
    return dict(y=y, x=x)


# ---- linear attention and layer norm ----


def _first_of(t, name, dims):
    if not isinstance(t, torch.Tensor) or t.dim() != dims or t.dtype not in _TYPES or not t.is_cuda:
        raise ValueError(f"{name}: expected a float32, bfloat16 or float16 device tensor of {dims} dimensions")
    if t.numel() == 0:
        raise ValueError(f"{name}: has no elements")
    return t.device, _TYPES[t.dtype]


def linear_bytes(op, dtype, Bsz, H, N, P, G, L, S=None, packed=False):
    """ssm_linear_bytes; dtype is a torch type"""
    out = ctypes.c_size_t()
    rc = lib.ssm_linear_bytes(int(op), _TYPES[dtype], int(Bsz), int(H), int(N), int(P), int(G), int(L),
                              int(Bsz if S is None else S), int(bool(packed)), ctypes.byref(out))
    if rc != OK:
        raise SSMError("ssm_linear_bytes", rc)
    return out.value


def _linear(q, k, v, g, beta, D, scale, x0):
    dev, code = _first_of(v, "v", 4)
    Bsz, H, P, L = v.shape
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q: expected [Bsz, G, N, L]")
    G, N = q.shape[1], q.shape[2]
    _activation(q, "q", v.dtype, (Bsz, G, N, L), dev)
    _activation(k, "k", v.dtype, (Bsz, G, N, L), dev)
    _activation(g, "g", torch.float32, (Bsz, H, L), dev)
    if beta is not None:
        _activation(beta, "beta", torch.float32, (Bsz, H, L), dev)
    _check(D, "D", torch.float32, (H,), dev)
    if x0 is not None and not isinstance(x0, torch.Tensor):
        raise ValueError("x0: expected a torch.float32 tensor")
    args = Linear(H, G, N, P, code, float(scale), _group_view(q), _group_view(k), _group_view(v), _view(g), _view(beta),
                  _address(D), _address(x0))
    return dev, Bsz, H, L, N, P, G, args


def linear_attention(q, k, v, g, beta=None, D=None, scale=1.0, x0=None, x_out=None, want_state=False, save=False,
                     offsets=None, lengths=None, slots=None, y=None, workspace=None):
    """ssm_linear_attention: x_t = exp(g_t) x_{t-1} + beta_t k_t v_t^T,
    y_t = scale x_t^T q_t + D v_t per head, over v [Bsz,H,P,L], q, k [Bsz,G,N,L]
    (shared by H/G heads), g, beta float32 [Bsz,H,L] (any strides, also of 0), D
    float32 [H].  x0: the states before the first step, float32 [S,H,N,P] (with
    slots, a pool [rows,H,N,P]); the states after the last go to x_out (which may
    be x0), or to a new tensor with want_state.  save keeps what
    linear_attention_backward needs.  offsets, lengths, slots as for
    selective_scan.  y is not written where no sequence runs, and not seen by
    autograd.  Returns dict(y, x, saved)."""
    dev, Bsz, H, L, N, P, G, args = _linear(q, k, v, g, beta, D, scale, x0)
    S = _count(Bsz, offsets)
    rows = _pool(_states(x0, "x0", torch.float32, S, slots, (H, N, P), dev),
                 _states(x_out, "x_out", torch.float32, S, slots, (H, N, P), dev), "x0 and x_out")
    if slots is not None and (save or (want_state and x_out is None)):
        raise ValueError("slots: give x_out, and no save")
    with _on(dev):
        if x_out is None and want_state:
            x_out = torch.empty((S, H, N, P), dtype=torch.float32, device=dev)
        seq = _sequences(Bsz, L, dev, offsets, lengths, slots, rows or _any_slot(H))
        if y is None:
            y = _like(v)
        else:
            _activation(y, "y", v.dtype, (Bsz, H, P, L), dev)
        sizes = (v.dtype, Bsz, H, N, P, G, L, S, offsets is not None)
        nbytes = linear_bytes(OP_LINEAR_ATTENTION, *sizes)
        ws = _scratch(nbytes, dev, workspace) if nbytes else None
        saved, sbytes = None, 0
        if save:
            sbytes = linear_bytes(OP_LINEAR_SAVED, *sizes)
            saved = torch.empty(sbytes, dtype=torch.uint8, device=dev)
        rc = lib.ssm_linear_attention(seq, args, _group_view(y), _address(x_out), _address(saved), sbytes, _address(ws),
                                      nbytes, _queue(dev))
    if rc != OK:
        raise SSMError("ssm_linear_attention", rc)
    return dict(y=y, x=x_out, saved=saved)


def linear_attention_backward(q, k, v, g, dy, beta=None, D=None, scale=1.0, x0=None, dx=None, saved=None, offsets=None,
                              lengths=None, workspace=None):
    """ssm_linear_attention_backward: gradients for dy [Bsz,H,P,L] of y and dx
    (float32 [S,H,N,P], or None) of the final states; the other arguments as in the
    forward call, saved from it (None: the states are computed again).  dg and
    dbeta are [Bsz,H,L] also where g and beta are broadcast.  Returns dict(dq, dk,
    dv, dg, dbeta, dD, dx0), None for the gradient of what was not given."""
    dev, Bsz, H, L, N, P, G, args = _linear(q, k, v, g, beta, D, scale, x0)
    _activation(dy, "dy", v.dtype, (Bsz, H, P, L), dev)
    with _on(dev):
        seq = _sequences(Bsz, L, dev, offsets, lengths, None, 0)
        S = seq.S
        _check(x0, "x0", torch.float32, (S, H, N, P), dev)
        _check(dx, "dx", torch.float32, (S, H, N, P), dev)
        sizes = (v.dtype, Bsz, H, N, P, G, L, S, offsets is not None)
        sbytes = linear_bytes(OP_LINEAR_SAVED, *sizes)
        if saved is None:
            saved = torch.empty(sbytes, dtype=torch.uint8, device=dev)
            nbytes = linear_bytes(OP_LINEAR_ATTENTION, *sizes)
            ws = _scratch(nbytes, dev, None) if nbytes else None
            rc = lib.ssm_linear_attention(seq, args, None, None, _address(saved), sbytes, _address(ws), nbytes, _queue(dev))
            if rc != OK:
                raise SSMError("ssm_linear_attention", rc)
        elif not (isinstance(saved, torch.Tensor) and saved.dtype == torch.uint8 and saved.device == dev
                  and saved.is_contiguous()):
            raise ValueError(f"saved: expected the uint8 tensor of the forward call on {dev}")
        whole = offsets is None and lengths is None
        dq, dk, dv = _like(q, whole), _like(k, whole), _like(v, whole)
        f32 = lambda *shape: (torch.empty if whole else torch.zeros)(shape, dtype=torch.float32, device=dev)  # noqa: E731
        dg, dbeta = f32(Bsz, H, L), f32(Bsz, H, L) if beta is not None else None
        dD, dx0 = f32(H) if D is not None else None, f32(S, H, N, P) if x0 is not None else None
        grads = LinearGrads(_group_view(dq), _group_view(dk), _group_view(dv), _view(dg), _view(dbeta), _address(dD),
                            _address(dx0))
        nbytes = linear_bytes(OP_LINEAR_ATTENTION_BACKWARD, *sizes)
        ws = _scratch(nbytes, dev, workspace)
        rc = lib.ssm_linear_attention_backward(seq, args, _address(saved), saved.numel(), _group_view(dy), _address(dx),
                                               grads, _address(ws), nbytes, _queue(dev))
    if rc != OK:
        raise SSMError("ssm_linear_attention_backward", rc)
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, dD=dD, dx0=dx0)


def linear_attention_step(q, k, v, g, x, beta=None, D=None, scale=1.0, slots=None, y=None):
    """ssm_linear_attention_step: one token per sequence, v [Bsz,H,P], q, k
    [Bsz,G,N], g, beta float32 [Bsz,H] (any strides); x float32 [Bsz,H,N,P] (with
    slots, a pool [rows,H,N,P]) moves on in place.  y's rows whose slot names no
    state are not written.  Returns dict(y, x)."""
    dev, code = _first_of(v, "v", 3)
    Bsz, H, P = v.shape
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: expected [Bsz, G, N]")
    G, N = q.shape[1], q.shape[2]
    _activation(q, "q", v.dtype, (Bsz, G, N), dev)
    _activation(k, "k", v.dtype, (Bsz, G, N), dev)
    _activation(g, "g", torch.float32, (Bsz, H), dev)
    if beta is not None:
        _activation(beta, "beta", torch.float32, (Bsz, H), dev)
    _check(D, "D", torch.float32, (H,), dev)
    _check(slots, "slots", torch.int32, (Bsz,), dev)
    if x is None:
        raise ValueError("x: needed")
    rows = _states(x, "x", torch.float32, Bsz, slots, (H, N, P), dev)
    with _on(dev):
        if y is None:
            y = torch.empty((Bsz, H, P), dtype=v.dtype, device=dev)
        else:
            _activation(y, "y", v.dtype, (Bsz, H, P), dev)
        args = LinearToken(Bsz, H, G, N, P, code, float(scale), _address(slots), rows, q.data_ptr(), k.data_ptr(),
                           v.data_ptr(), y.data_ptr(), g.data_ptr(), _address(beta), *_strides(q), *_strides(k),
                           *_strides(v), *_strides(y), *_strides(g), *((0, 0) if beta is None else _strides(beta)),
                           _address(D), x.data_ptr())
        rc = lib.ssm_linear_attention_step(args, _queue(dev))
    if rc != OK:
        raise SSMError("ssm_linear_attention_step", rc)
    return dict(y=y, x=x)


def _steps_of(t):
    """[Bsz,H] as [Bsz,H,1]"""
    return t.unsqueeze(-1) if isinstance(t, torch.Tensor) and t.dim() == 2 else t


def _norm(u, weight, bias, z, gate, rms, groups, eps):
    if gate not in GATES:
        raise ValueError("gate: expected 'before' or 'after'")
    if isinstance(u, torch.Tensor) and u.dim() == 2:
        u, z = _steps_of(u), _steps_of(z)
    dev, code = _first(u, 3)
    Bsz, H, L = u.shape
    if z is not None:
        _activation(z, "z", u.dtype, (Bsz, H, L), dev)
    _check(weight, "weight", torch.float32, (H,), dev)
    _check(bias, "bias", torch.float32, (H,), dev)
    args = Norm(Bsz, H, L, int(groups), code, int(bool(rms)), 0 if z is None else GATES[gate], float(eps), _view(u),
                _view(z), _address(weight), _address(bias))
    return dev, u, args


def layer_norm(u, weight=None, bias=None, z=None, gate="after", rms=False, groups=1, eps=1e-5, y=None):
    """ssm_layer_norm: over the channels of each of `groups` groups of u [Bsz,H,L]
    (or [Bsz,H], one token each), y = n weight + bias with n = (u - mean) /
    sqrt(var + eps), or with rms u / sqrt(mean u^2 + eps); weight, bias float32 [H].
    z (like u) gates with silu(z): the result (gate "after") or u itself
    ("before").  y must not overlap u or z.  Not seen by autograd.  Returns dict(y)."""
    dev, steps, args = _norm(u, weight, bias, z, gate, rms, groups, eps)
    with _on(dev):
        if y is None:
            out = _like(steps)
            y = out.squeeze(-1) if u.dim() == 2 else out
        else:
            _activation(y, "y", u.dtype, tuple(u.shape), dev)
            out = _steps_of(y)
        rc = lib.ssm_layer_norm(args, _view(out), _queue(dev))
    if rc != OK:
        raise SSMError("ssm_layer_norm", rc)
    return dict(y=y)


def layer_norm_backward(u, dy, weight=None, bias=None, z=None, gate="after", rms=False, groups=1, eps=1e-5,
                        workspace=None):
    """ssm_layer_norm_backward: gradients for dy of y, the other arguments as in
    the forward call (whose results are not needed).  Returns dict(du, dz, dweight,
    dbias), None for the gradient of what was not given."""
    dev, steps, args = _norm(u, weight, bias, z, gate, rms, groups, eps)
    _activation(dy, "dy", u.dtype, tuple(u.shape), dev)
    Bsz, H, L = steps.shape
    with _on(dev):
        du = _like(steps)
        dz = _like(_steps_of(z)) if z is not None else None
        f32 = lambda t: torch.empty((H,), dtype=torch.float32, device=dev) if t is not None else None  # noqa: E731
        dweight, dbias = f32(weight), f32(bias)
        ws, nbytes = None, 0
        if weight is not None or bias is not None:
            size = ctypes.c_size_t()
            rc = lib.ssm_layer_norm_bytes(Bsz, H, L, int(groups), ctypes.byref(size))
            if rc != OK:
                raise SSMError("ssm_layer_norm_bytes", rc)
            nbytes = size.value
            ws = _scratch(nbytes, dev, workspace)
        rc = lib.ssm_layer_norm_backward(args, _view(_steps_of(dy)), _view(du), _view(dz), _address(dweight),
                                         _address(dbias), _address(ws), nbytes, _queue(dev))
    if rc != OK:
        raise SSMError("ssm_layer_norm_backward", rc)
    if u.dim() == 2:
        du, dz = du.squeeze(-1), None if dz is None else dz.squeeze(-1)
    return dict(du=du, dz=dz, dweight=dweight, dbias=dbias)


def to_device(params, device="cuda:0"):
    """Move an inputs.Params (numpy) to torch device tensors (a plain copy)."""
    f = lambda a: torch.from_numpy(a).to(device)
    return dict(Lambda=f(params.Lambda), P=f(params.P), Q=f(params.Q), B=f(params.B), C=f(params.C),
                dt=f(params.dt), D=f(params.D))
