"""Refusals of the linear, gated and gated-norm entry points on the host, before
any HIP call (CPU): no call here launches a kernel."""
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


def _linear(lib, x=at(0), w=at(1), b=at(2), r=at(3), pre=at(4), y=at(5), rows=4, K=64, N=24, act=1, alpha=1.0,
            dtype=0):
    return lib.gla_linear(x, w, b, r, pre, y, rows, K, N, act, alpha, dtype, None)


def test_linear_refusals(lib):
    f = lambda **kw: _linear(lib, **kw)
    assert f(x=None) == A and f(w=None) == A and f(y=None) == A
    for name, i in (("x", 0), ("w", 1), ("b", 2), ("r", 3), ("pre", 4), ("y", 5)):
        assert f(**{name: at(i, 8)}) == A
    assert f(rows=-1) == A and f(K=-8) == A and f(N=-8) == A and f(dtype=2) == A and f(act=4) == A and f(act=-1) == A
    assert f(K=60) == U and f(N=20) == U and f(K=0) == U and f(N=65544) == U and f(K=65544) == U
    assert f(rows=(1 << 31) + 1) == U
    # outputs over inputs or each other, in whole or in part
    assert f(y=at(0)) == A and f(y=at(1, 16)) == A and f(y=at(2)) == A and f(y=at(4)) == A
    assert f(pre=at(3)) == A and f(pre=at(0, 16)) == A and f(y=at(3, 16)) == A
    assert f(y=at(0, 4 * 64 * 2 - 16)) == A
    assert f(rows=0, x=None) == OK and f(N=0, x=None) == OK and f(rows=0, K=0, x=None) == OK


def _linear_bwd(lib, x=at(0), w=at(1), pre=at(2), gy=at(3), gx=at(4), gw=at(5), gb=at(6), rows=4, K=64, N=24, act=1,
                dtype=0, ws=at(7), nws=10 ** 9):
    return lib.gla_linear_bwd(x, w, pre, gy, gx, gw, gb, rows, K, N, act, 1.0, dtype, ws, nws, None)


def test_linear_backward_refusals(lib):
    f = lambda **kw: _linear_bwd(lib, **kw)
    assert f(x=None) == A and f(w=None) == A and f(pre=None) == A and f(gy=None) == A
    for name, i in (("x", 0), ("w", 1), ("pre", 2), ("gy", 3), ("gx", 4), ("gw", 5), ("gb", 6)):
        assert f(**{name: at(i, 8)}) == A
    assert f(rows=-1) == A and f(dtype=5) == A and f(act=9) == A and f(K=60) == U and f(K=0) == U and f(N=12) == U
    assert f(ws=None) == A and f(ws=at(7, 64)) == A and f(nws=0) == W
    need = lib.gla_linear_bwd_workspace_bytes(4, 64, 24, 1, 0)
    assert need > 0 and f(nws=need - 1) == W
    for i in range(4):
        assert f(gx=at(i)) == A and f(gw=at(i)) == A and f(gb=at(i)) == A
    assert f(gx=at(5)) == A and f(gb=at(4)) == A and f(gw=at(7)) == A
    # what is not wanted is not looked at
    assert f(gx=None, w=None, nws=0) == W and f(gw=None, x=None, nws=0) == W
    assert f(act=0, pre=None, nws=0) == W
    assert f(gx=None, gw=None, gb=None, gy=None) == OK
    assert f(rows=0, gy=None) == OK and f(N=0, gy=None) == OK
    n = lib.gla_linear_bwd_workspace_bytes
    assert n(0, 64, 24, 1, 0) == 0 and n(4, 60, 24, 1, 0) == 0 and n(4, 64, 24, 7, 0) == 0 and n(4, 64, 24, 0, 0) > 0


def _ff(lib, x=at(0), wg=at(1), wu=at(2), a=at(3), u=at(4), h=at(5), rows=4, K=64, F=24, act=1, dtype=0):
    return lib.gla_gated_ff(x, wg, wu, a, u, h, rows, K, F, act, dtype, None)


def test_gated_ff_refusals(lib):
    f = lambda **kw: _ff(lib, **kw)
    assert f(x=None) == A and f(wg=None) == A and f(wu=None) == A and f(h=None) == A
    for name, i in (("x", 0), ("wg", 1), ("wu", 2), ("a", 3), ("u", 4), ("h", 5)):
        assert f(**{name: at(i, 2)}) == A
    assert f(rows=-2) == A and f(dtype=3) == A and f(act=5) == A and f(K=12) == U and f(F=12) == U and f(K=0) == U
    assert f(h=at(0)) == A and f(a=at(1)) == A and f(u=at(2)) == A and f(a=at(4)) == A and f(h=at(3)) == A
    assert f(rows=0, x=None) == OK and f(F=0, x=None) == OK


def _ff_bwd(lib, x=at(0), wg=at(1), wu=at(2), a=at(3), u=at(4), gh=at(5), gx=at(6), gg=at(7), gu=at(8), rows=4, K=64,
            F=24, act=1, dtype=0, ws=at(9), nws=10 ** 9):
    return lib.gla_gated_ff_bwd(x, wg, wu, a, u, gh, gx, gg, gu, rows, K, F, act, dtype, ws, nws, None)


def test_gated_ff_backward_refusals(lib):
    f = lambda **kw: _ff_bwd(lib, **kw)
    for name, i in (("x", 0), ("wg", 1), ("wu", 2), ("a", 3), ("u", 4), ("gh", 5)):
        assert f(**{name: None}) == A and f(**{name: at(i, 4)}) == A
    assert f(gx=at(6, 8)) == A and f(gg=at(7, 8)) == A and f(gu=at(8, 8)) == A
    assert f(gg=None) == A and f(gu=None) == A  # one without the other
    assert f(ws=None) == A and f(ws=at(9, 32)) == A and f(nws=0) == W and f(K=4) == U and f(act=-1) == A
    for i in range(6):
        assert f(gx=at(i)) == A and f(gg=at(i)) == A and f(gu=at(i)) == A
    assert f(gx=at(7)) == A and f(gg=at(8)) == A and f(gu=at(9)) == A
    assert f(gx=None, wg=None, wu=None, nws=0) == W and f(gg=None, gu=None, x=None, nws=0) == W
    assert f(gx=None, gg=None, gu=None, gh=None) == OK and f(rows=0, gh=None) == OK
    n = lib.gla_gated_ff_bwd_workspace_bytes
    assert n(4, 64, 24, 0) >= 2 * 4 * 24 * 2 and n(0, 64, 24, 0) == 0 and n(4, 64, 20, 0) == 0


def _norm(lib, x=at(0), r=at(1), post=at(2), gate=at(3), groups=2, scale=at(4), w=at(5), eps=1e-6, s=at(6), y=at(7),
          rows=4, F=64, dtype=0):
    return lib.gla_gated_add_rmsnorm(x, r, post, gate, groups, scale, w, eps, s, y, rows, F, dtype, None)


def test_gated_norm_refusals(lib):
    f = lambda **kw: _norm(lib, **kw)
    assert f(x=None) == A and f(r=None) == A and f(w=None) == A and f(y=None) == A
    for name, i in (("x", 0), ("r", 1), ("post", 2), ("gate", 3), ("scale", 4), ("w", 5), ("s", 6), ("y", 7)):
        assert f(**{name: at(i, 4)}) == A
    assert f(rows=-1) == A and f(F=-8) == A and f(dtype=4) == A and f(eps=-1.0) == A and f(eps=float("nan")) == A
    assert f(F=60) == U and f(F=16392) == U and f(rows=(1 << 31) + 1) == U
    assert f(groups=0) == A and f(groups=3) == A and f(groups=8) == A and f(groups=-1) == A
    assert f(y=at(6)) == A and f(s=at(2)) == A and f(y=at(3)) == A and f(y=at(5)) == A
    assert f(s=at(0, 16)) == A and f(y=at(1, 16)) == A and f(s=at(0), y=at(0)) == A
    assert f(rows=0, x=None) == OK and f(F=0, x=None) == OK and f(rows=0, gate=None, groups=0) == OK


def _norm_bwd(lib, x=at(0), s=at(1), post=at(2), gate=at(3), groups=2, scale=at(4), w=at(5), eps=1e-6, gy=at(6),
              gs=at(7), gx=at(8), gr=at(9), gp=at(10), gg=at(11), gsc=at(12), gw=at(13), rows=4, F=64, dtype=0,
              ws=at(14), nws=10 ** 9):
    return lib.gla_gated_add_rmsnorm_bwd(x, s, post, gate, groups, scale, w, eps, gy, gs, gx, gr, gp, gg, gsc, gw, rows,
                                         F, dtype, ws, nws, None)


def test_gated_norm_backward_refusals(lib):
    f = lambda **kw: _norm_bwd(lib, **kw)
    for name in ("x", "s", "w", "gy", "gx", "gr", "gw", "ws"):
        assert f(**{name: None}) == A
    for i, name in enumerate(("x", "s", "post", "gate", "scale", "w", "gy", "gs", "gx", "gr", "gp", "gg", "gsc", "gw")):
        j = {"w": 5, "gy": 6, "gs": 7}.get(name, i)
        assert f(**{name: at(j, 8)}) == A
    assert f(groups=3) == A and f(groups=0) == A and f(F=60) == U and f(eps=-1.0) == A and f(dtype=2) == A
    assert f(post=None) == A and f(gate=None) == A and f(scale=None) == A  # gradients of what is not there
    assert f(nws=0) == W and f(ws=at(14, 128)) == A
    for i in range(8):
        for name in ("gp", "gg", "gsc", "gw"):
            assert f(**{name: at(i)}) == A
    for i in (2, 3, 4, 5):
        assert f(gx=at(i)) == A and f(gr=at(i)) == A
    assert f(gx=at(9)) == A and f(gp=at(8)) == A and f(gw=at(14)) == A and f(gx=at(0, 16)) == A and f(gr=at(6, 16)) == A
    for i in (0, 1, 6, 7):  # row for row: only the workspace's size is wrong
        assert f(gx=at(i), nws=0) == W and f(gr=at(i), nws=0) == W
    assert f(rows=0, x=None) == OK and f(gp=None, gg=None, gsc=None, nws=0) == W
    n = lib.gla_gated_add_rmsnorm_bwd_workspace_bytes
    assert n(4, 2, 64) > 0 and n(4, 3, 64) == 0 and n(0, 1, 64) == 0 and n(4, 1, 60) == 0 and n(4, 0, 64) == 0


