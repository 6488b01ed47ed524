"""Refusals of the gradient, single-token and norm entry points on the host,
before any HIP call (CPU): no call here launches a kernel."""
import ctypes
import os

import pytest

from recurrent_vision_token_gla_amd import gla

A, U, W, OK = gla.E_ARG, gla.E_UNSUPPORTED, gla.E_WORKSPACE, gla.OK
P = 0x100000  # 256-aligned, never dereferenced
MIB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gla.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return gla.load()


def at(i, off=0):
    """The i-th of a row of fake buffers, 1 MiB apart."""
    return P + i * MIB + off


def _bwd(lib, q=at(0), go=at(4), gq=at(5), gkey=at(6), gv=at(7), ggk=at(8), s0=None, gsf=None,
         gs0=None, B=1, H=2, gh=4, gw=5, dk=32, dv=64, dirs=(0,), dtype=0, ws=at(9), nws=10 ** 9):
    arr = (ctypes.c_int32 * max(1, len(dirs)))(*dirs) if dirs is not None else None
    return lib.gla_bwd(q, at(1), at(2), at(3), go, gq, gkey, gv, ggk, B, H, gh, gw, dk, dv, arr,
                       dtype, s0, gsf, gs0, ws, nws, None)


def test_bwd_refusals(lib):
    assert _bwd(lib, q=None) == A and _bwd(lib, go=None) == A and _bwd(lib, ggk=None) == A
    assert _bwd(lib, q=at(0, 8)) == A and _bwd(lib, gv=at(7, 2)) == A  # misaligned
    assert _bwd(lib, B=-1) == A and _bwd(lib, gw=-2) == A and _bwd(lib, dtype=2) == A
    assert _bwd(lib, dk=48) == U and _bwd(lib, dv=128) == U and _bwd(lib, H=70000) == U
    assert _bwd(lib, dirs=None) == A and _bwd(lib, dirs=(4,)) == A
    assert _bwd(lib, s0=at(10, 4)) == A and _bwd(lib, gs0=at(10, 8)) == A
    assert _bwd(lib, ws=None) == A and _bwd(lib, ws=at(9, 16)) == A
    need = gla.bwd_workspace_bytes(1, 2, 4, 5, 32, 64)
    assert need > 0 and _bwd(lib, nws=need - 1) == W
    # outputs over inputs, over each other, over the workspace, in whole or in part
    rows = 4 * 5 * 2
    assert _bwd(lib, gq=at(0)) == A and _bwd(lib, gq=at(0, rows * 32 * 2 - 16)) == A
    assert _bwd(lib, gv=at(4)) == A and _bwd(lib, gkey=at(5)) == A and _bwd(lib, ggk=at(9)) == A
    assert _bwd(lib, gsf=at(10), gs0=at(10, 16)) == A      # beside itself
    assert _bwd(lib, s0=at(10), gs0=at(10)) == A           # s0 is still read
    assert _bwd(lib, gs0=at(9, 256)) == A
    # every check above comes before the workspace's size; these pass them all
    assert _bwd(lib, gsf=at(10), gs0=at(10), nws=0) == W
    assert _bwd(lib, gq=at(0, rows * 32 * 2), nws=0) == W
    # empty problems look at nothing
    assert _bwd(lib, q=None, B=0, dirs=None) == OK and _bwd(lib, q=None, gh=0, ws=None) == OK
    assert gla.bwd_workspace_bytes(0, 2, 4, 5, 32, 64) == 0
    assert gla.bwd_workspace_bytes(1, 2, 4, 5, 33, 64) == 0
    # S and D (float [dk][dv]) and the decays, per (batch, head, chunk)
    assert gla.bwd_workspace_bytes(2, 3, 9, 15, 64, 64) == 2 * 3 * 3 * (2 * 64 * 64 + 64) * 4


def _step(lib, q=at(0), o=at(4), state=at(5), slots=at(6), n=8, B=4, H=2, dk=32, dv=64, dtype=0,
          gated=False, gate=at(7), w=at(8), eps=1e-6):
    if not gated:
        return lib.gla_step(q, at(1), at(2), at(3), o, B, H, dk, dv, dtype, state, n, slots, None)
    return lib.gla_step_gated(q, at(1), at(2), at(3), gate, w, eps, o, B, H, dk, dv, dtype, state, n,
                              slots, None)


def test_step_refusals(lib):
    for gated in (False, True):
        f = lambda **kw: _step(lib, gated=gated, **kw)
        assert f(q=None) == A and f(o=None) == A and f(state=None) == A
        assert f(q=at(0, 4)) == A and f(state=at(5, 8)) == A and f(slots=at(6, 2)) == A
        assert f(B=-1) == A and f(n=-1) == A and f(dtype=3) == A
        assert f(dk=16) == U and f(dv=96) == U and f(B=65536) == U and f(H=65536) == U
        assert f(slots=None, n=3) == A                      # four rows, three states
        assert f(o=at(0)) == A and f(o=at(5)) == A          # over an input, over the states
        assert f(state=at(6), n=1) == A                     # the slots inside the states
        assert f(B=0, q=None) == OK and f(H=0, q=None) == OK
    assert _step(lib, gated=True, gate=None) == A and _step(lib, gated=True, w=None) == A
    assert _step(lib, gated=True, gate=at(7, 8)) == A and _step(lib, gated=True, w=at(8, 4)) == A
    assert _step(lib, gated=True, eps=-1.0) == A and _step(lib, gated=True, eps=float("nan")) == A
    assert _step(lib, gated=True, o=at(7)) == A


def _norm(lib, x=at(0), r=at(1), w=at(2), eps=1e-6, s=at(3), y=at(4), rows=4, F=64, dtype=0, q8=False,
          sc=at(5)):
    if q8:
        return lib.gla_add_rmsnorm_q8(x, r, w, eps, s, y, sc, rows, F, dtype, None)
    return lib.gla_add_rmsnorm(x, r, w, eps, s, y, rows, F, dtype, None)


def test_norm_refusals(lib):
    for q8 in (False, True):
        f = lambda **kw: _norm(lib, q8=q8, **kw)
        assert f(x=None) == A and f(w=None) == A and f(y=None) == A
        assert f(x=at(0, 8)) == A and f(r=at(1, 2)) == A and f(s=at(3, 4)) == A and f(w=at(2, 4)) == A
        assert f(rows=-1) == A and f(F=-8) == A and f(dtype=7) == A and f(eps=-1e-6) == A
        assert f(F=60) == U and f(F=16392) == U and f(rows=(1 << 31) + 1) == U
        assert f(y=at(3)) == A and f(y=at(2)) == A          # over the sum, over the weight
        assert f(s=at(0, 16)) == A and f(y=at(1, 16)) == A  # over an input in part
        assert f(rows=0, x=None) == OK and f(F=0, x=None) == OK
    assert _norm(lib, q8=True, sc=None) == A and _norm(lib, q8=True, sc=at(5, 2)) == A
    assert _norm(lib, q8=True, y=at(0)) == A and _norm(lib, q8=True, sc=at(1)) == A
    assert _norm(lib, s=at(0), y=at(0)) == A


def _norm_bwd(lib, s=at(0), w=at(1), eps=1e-6, gy=at(2), gs=None, gx=at(3), gw=at(4), rows=4, F=64,
              dtype=0, ws=at(5), nws=10 ** 9):
    return lib.gla_add_rmsnorm_bwd(s, w, eps, gy, gs, gx, gw, rows, F, dtype, ws, nws, None)


def test_norm_backward_refusals(lib):
    f = lambda **kw: _norm_bwd(lib, **kw)
    assert f(s=None) == A and f(gy=None) == A and f(gx=None) == A and f(gw=None) == A and f(w=None) == A
    assert f(gs=at(6, 8)) == A and f(gw=at(4, 4)) == A and f(eps=-1.0) == A
    assert f(F=60) == U and f(rows=-1) == A and f(dtype=2) == A
    assert f(ws=None) == A and f(ws=at(5, 64)) == A and f(nws=0) == W
    assert f(gx=at(0, 16)) == A and f(gx=at(1)) == A and f(gx=at(4)) == A and f(gx=at(5)) == A
    assert f(gw=at(2)) == A and f(gw=at(1)) == A
    assert f(gx=at(0), nws=0) == W and f(gx=at(2), nws=0) == W  # in place: only the size is wrong
    assert f(rows=0, s=None) == OK
    n = lib.gla_add_rmsnorm_bwd_workspace_bytes
    assert n(4, 64) >= 64 * 4 and n(0, 64) == 0 and n(4, 60) == 0 and n(-1, 64) == 0


def _gate_bwd(lib, o=at(0), z=at(1), w=at(2), eps=1e-6, gy=at(3), go=at(4), gz=at(5), gw=at(6), rows=4,
              dv=64, dtype=0, ws=at(7), nws=10 ** 9):
    return lib.gla_gate_bwd(o, z, w, eps, gy, go, gz, gw, rows, dv, dtype, ws, nws, None)


def test_gate_backward_refusals(lib):
    f = lambda **kw: _gate_bwd(lib, **kw)
    for name in ("o", "z", "w", "gy", "go", "gz", "gw", "ws"):
        assert f(**{name: None}) == A
    assert f(o=at(0, 2)) == A and f(gw=at(6, 4)) == A and f(eps=-1.0) == A
    assert f(dv=48) == U and f(rows=-1) == A and f(dtype=2) == A and f(nws=0) == W
    assert f(go=at(0)) == A and f(gz=at(4)) == A and f(gw=at(7)) == A and f(go=at(3)) == A
    assert f(rows=0, o=None) == OK
    n = lib.gla_gate_bwd_workspace_bytes
    assert n(4, 64) >= 64 * 4 and n(0, 64) == 0 and n(4, 40) == 0
