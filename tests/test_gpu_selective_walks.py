"""The selective scan where a workgroup takes many tiles: whole sequences of several
tiles, chunks of four, sequences of thousands of steps, and gradients summed over many
workgroups of a group; against the float64 oracle, within bounds that are carried
through the recurrence (tests/selective_bounds.py).  Which form a size takes is
checked by the workspace it asks for."""
import numpy as np
import pytest

import oracle.selective_oracle as S
from tests import selective_bounds as T
from tests import selective_cases as K
from tests.test_gpu_selective import _f32, _int, _np, _scan_args, _ssm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ORDERS = [("f32", "rows"), ("bf16", "tokens"), ("f32", "mixed"), ("f16", "sliced")]


def _up256(n):
    return (n + 255) // 256 * 256


def _chunk_bytes(items, S_, H, N):
    """Workspace of a forward call in so many chunks: their ends and sums, and the start states."""
    Np = 16 if N <= 16 else 32 if N <= 32 else 64
    return _up256(items * H * Np * 4) + _up256(items * H * 4) + _up256(S_ * H * Np * 4)


def _check(a, name, order, spans, backward=True, **kw):
    ssm = _ssm()
    H, N = a["A"].shape
    rng = np.random.default_rng(91)
    dy = K.rounded(rng.standard_normal(a["u"].shape), name) if backward else None
    dl = K.rounded(rng.standard_normal((len(spans), H, N)), "f32") if backward else None
    err = T.scan_bounds(a, spans, dy, dl)
    args, more = _scan_args(a, name, order)
    f = ssm.selective_scan(*args, **more, want_state=True, save=backward, **kw)
    want, last, _ = K.oracle_scan(a, spans)
    T.within(_np(f["y"]), want, err["y"], name, "y")
    T.within(_np(f["x"]), last, err["x"], "f32", "x")
    if not backward:
        return
    out = ssm.selective_scan_backward(*args, K.on_device(dy, name, order), **more, dx=_f32(dl), saved=f["saved"], **kw)
    want = K.oracle_scan_grad(a, dy, dl, spans)
    for k, v in out.items():
        if v is not None:
            T.within(_np(v), want[k], err[k], name if k in ("du", "ddelta", "dz", "dB", "dC") else "f32", k)


@pytest.mark.parametrize("name,order", ORDERS)
@pytest.mark.parametrize("N", [16, 20, 40])
def test_whole_sequences_of_many_tiles(name, order, N):
    # 171 rows: two chunks would not pay, so a workgroup takes five tiles and a part of one
    Bsz, H, L = 171, 4, 170
    assert _ssm().selective_bytes(_ssm().OP_SELECTIVE_SCAN, Bsz, H, N, 1, L) == 0
    a = K.scan_inputs(92, name, Bsz, H, L, N, state=True)
    _check(a, name, order, S.dense_spans(Bsz, L))


@pytest.mark.parametrize("name,order", ORDERS)
@pytest.mark.parametrize("N", [16, 24, 40])
def test_chunks_of_four_tiles(name, order, N):
    Bsz, H, L = 86, 4, 400     # 128, 128, 128 and 16 steps
    assert _ssm().selective_bytes(_ssm().OP_SELECTIVE_SCAN, Bsz, H, N, 1, L) == _chunk_bytes(4 * Bsz, Bsz, H, N)
    a = K.scan_inputs(93, name, Bsz, H, L, N, state=True)
    _check(a, name, order, S.dense_spans(Bsz, L))


@pytest.mark.parametrize("name,order", ORDERS)
def test_ragged_walks(name, order):
    Bsz, H, L, N = 171, 4, 170, 16
    r = np.random.default_rng(94)
    lens = [int(v) for v in r.integers(0, L + 1, Bsz)]
    lens[:6] = [0, 1, 31, 32, 33, 170]
    a = K.scan_inputs(95, name, Bsz, H, L, N, state=True)
    _check(a, name, order, S.dense_spans(Bsz, L, lens), lengths=_int(lens))


@pytest.mark.parametrize("name,order", [("f32", "rows"), ("f32", "tokens"), ("bf16", "tokens")])
def test_thousands_of_steps(name, order):
    # chunks of two tiles, 256 of them
    a = K.scan_inputs(96, name, 1, 3, 16384, 16, state=True)
    _check(a, name, order, S.dense_spans(1, 16384), backward=False)
    a = K.scan_inputs(97, name, 1, 3, 4000, 16, state=True)
    _check(a, name, order, S.dense_spans(1, 4000))
    # packed, of 7, 2493, 0 and 1500 steps
    offs = [0, 7, 2500, 2500, 4000]
    a = K.scan_inputs(98, name, 1, 3, 4000, 16, state=True, S_=4)
    _check(a, name, order, S.packed_spans(offs), offsets=_int(offs))


@pytest.mark.parametrize("name,order", [("f32", "rows"), ("bf16", "tokens"), ("f16", "mixed")])
@pytest.mark.parametrize("H,G,N", [(1100, 1, 16), (2120, 2, 16), (1100, 1, 24), (1030, 1, 40)])
def test_gradients_over_many_workgroups(name, order, H, G, N):
    # 17 or 18 workgroups of a group: their rows of dB and dC are added 16 together, then one by one
    Bsz, L = 2, 40
    a = K.scan_inputs(99, name, Bsz, H, L, N, G, state=True)
    _check(a, name, order, S.dense_spans(Bsz, L))
