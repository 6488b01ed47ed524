"""GPU: weight gradients of the norm and of the output gate held to the tree
their sums are taken in, at sizes where every workgroup takes several rows; and
the recurrence's serial scan with float states.

Bounds, u = 2^-24 of the sum of magnitudes over R rows. A thread adds the rows
it walks one after the other, at most ceil(steps / 1024) of them; up to four
rows of a workgroup are joined (3 u), or the lanes and waves of one (6 u); then
at most 16, 8 and 8 partial sums: 32 u. A term itself is off by (F/64 + 24) u
(the row's norm), or (32 + 2 |z|) u in the gate (exp's argument is rounded once).
So one row of R that is left out, or taken twice, is outside: it moves the sum by
2^24 / R u on average, 254 u of the 66,001 rows that are held to 78 u here, and
every test checks that its bound is below a third of an average row."""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_bwd
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


def steps(rows, per):
    return -(-(-(-rows // per)) // 1024)


def held(name, got, want, mag, units, rows):
    got = got.double().cpu().numpy()
    assert units * U < 1 / (3 * rows)
    worst = float(np.max(np.abs(got - want) / (units * U * mag)))
    say(f"{name}: {worst:.3f} of {units:.0f} u")
    assert worst <= 1


@pytest.mark.parametrize("rows,F", [(4500, 64), (5000, 768), (1500, 2056), (2500, 1536), (1100, 4104), (1030, 8200)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_norm_weight_gradient(rows, F, dtype):
    r = np.random.default_rng(rows + F)
    s, gy = (r.standard_normal((rows, F)).astype(dtype) for _ in range(2))
    w = (1 + 0.1 * r.standard_normal(F)).astype(np.float32)
    gx, gw = gla.add_rmsnorm_bwd(*to_dev(s, w), EPS, *to_dev(gy))
    torch.cuda.synchronize()
    want, ww = oracle.add_rmsnorm_backward(s, w, EPS, gy)
    s, gy = s.astype(np.float64), gy.astype(np.float64)
    rstd = 1 / np.sqrt(np.mean(s * s, 1, keepdims=True) + EPS)
    units = steps(rows, 4 if F <= 1024 else 1) + 3 + 32 + F / 64 + 24
    held(f"norm {rows}x{F} {np.dtype(dtype).name}", gw, ww, np.sum(np.abs(gy * s * rstd), 0), units, rows)
    # the rows themselves, all of them
    gn, n = gy * w, s * rstd
    tol = (2 * F / 64 + 32) * U * rstd * (np.abs(gn) + np.abs(n) * np.mean(np.abs(gn * n), 1, keepdims=True))
    tol += 2.0 ** -11 * np.abs(want) + 2.0 ** -25 if dtype == np.float16 else U * np.abs(want)
    assert float(np.max(np.abs(gx.double().cpu().numpy() - want) / tol)) <= 1


@pytest.mark.parametrize("rows,dv", [(38400, 64), (33000, 64), (66001, 32)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_gate_weight_gradient(rows, dv, dtype):
    r = np.random.default_rng(rows + dv)
    o, gy = (r.standard_normal((rows, dv)).astype(dtype) for _ in range(2))
    z = np.clip(r.standard_normal((rows, dv)), -3, 3).astype(dtype)
    w = (1 + 0.1 * r.standard_normal(dv)).astype(np.float32)
    _, _, gw = gla.gate_bwd(*to_dev(o, z, w), EPS, *to_dev(gy))
    torch.cuda.synchronize()
    want = oracle.rmsnorm_gate_backward(o, z, w, EPS, gy)[2]
    o, z, gy = (a.astype(np.float64) for a in (o, z, gy))
    n = o / np.sqrt(np.mean(o * o, 1, keepdims=True) + EPS)
    units = steps(rows, 256 // (dv // 8)) + 6 + 32 + 32 + 2 * 3
    held(f"gate {rows}x{dv} {np.dtype(dtype).name}", gw, want, np.sum(np.abs(gy * n * oracle.silu(z)), 0), units, rows)


@pytest.mark.parametrize("chunks", [3, 8, 19])
def test_serial_scan_of_float_states(chunks):
    """25 chains of 64/64 are 25,600 groups of four state elements, enough for
    the scan that walks a chain in order: fewer chunks than its window of eight,
    one window, two and a rest."""
    T = 64 * chunks - 5
    x, s0, gsf = test_gpu_bwd.inputs(5, 1, T, 5, 64, 64, np.float32, 700 + chunks, carry=True)
    test_gpu_bwd.check(x, 1, T, [0, 1, 0, 1, 0], s0, gsf)
