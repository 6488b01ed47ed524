"""The gradient oracle against central differences of the forward oracle, and
its norms against hand-derived cases (CPU).

A central difference of a loss f with step h is off by h^2 f'''/6 + eps |f| / h:
with h = 1e-4, values of order one and float64 that is about 1e-8 relative; the
bar is 1e-6 of the largest gradient."""
import numpy as np
import pytest

import oracle

BAR, H = 1e-6, 1e-4


def _close(got, want):
    assert np.max(np.abs(got - want)) <= BAR * max(1.0, np.max(np.abs(want)))


def _differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + H
        up = f()
        x[i] = keep - H
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * H)
    return g


@pytest.mark.parametrize("dirs", [(0, 1), (2, 3)])
@pytest.mark.parametrize("carry", [False, True])
def test_recurrence_gradient_matches_differences(dirs, carry):
    rng = np.random.default_rng(71)
    B, gh, gw, Hh, dk, dv = 2, 2, 3, 2, 3, 2
    T = gh * gw
    x = {n: rng.standard_normal((B, T, Hh, d)) for n, d in (("q", dk), ("k", dk), ("v", dv))}
    x["gk"] = -rng.random((B, T, Hh, dk))
    go = rng.standard_normal((B, T, Hh, dv))
    s0 = rng.standard_normal((B, Hh, dk, dv)) if carry else None
    gsf = rng.standard_normal((B, Hh, dk, dv)) if carry else None

    def loss():
        o, sT = oracle.gla_forward(x["q"], x["k"], x["v"], x["gk"], gh, gw, dirs, impl="numpy",
                                   s0=s0, return_state=True)
        return float(np.sum(o * go) + (np.sum(sT * gsf) if carry else 0.0))

    grads = oracle.gla_backward(x["q"], x["k"], x["v"], x["gk"], go, gh, gw, dirs, s0, gsf)
    for g, n in zip(grads, ("q", "k", "v", "gk")):
        _close(g, _differences(loss, x[n]))
    if carry:
        _close(grads[4], _differences(loss, s0))


def test_recurrence_gradient_segments_agree():
    rng = np.random.default_rng(72)
    q, k, g = (rng.standard_normal((1, 23, 2, 4)) for _ in range(3))
    v, go = (rng.standard_normal((1, 23, 2, 3)) for _ in range(2))
    a = oracle.recurrence_backward(q, k, v, -np.abs(g), go, segment=64)
    b = oracle.recurrence_backward(q, k, v, -np.abs(g), go, segment=5)
    for x, y in zip(a, b):
        assert np.max(np.abs(x - y)) <= 1e-12


def test_gate_gradient_matches_differences():
    rng = np.random.default_rng(73)
    o, z, gy = (rng.standard_normal((3, 2, 4)) for _ in range(3))
    w = 1 + 0.1 * rng.standard_normal(4)
    grads = oracle.rmsnorm_gate_backward(o, z, w, 1e-3, gy)
    loss = lambda: float(np.sum(oracle.rmsnorm_gate(o, z, w, 1e-3) * gy))
    for g, x in zip(grads, (o, z, w)):
        _close(g, _differences(loss, x))


def test_norm_gradient_matches_differences():
    rng = np.random.default_rng(74)
    s, gy, gs = (rng.standard_normal((5, 8)) for _ in range(3))
    w = 1 + 0.1 * rng.standard_normal(8)
    gx, gw = oracle.add_rmsnorm_backward(s, w, 1e-3, gy, gs)
    loss = lambda: float(np.sum(oracle.add_rmsnorm(s, None, w, 1e-3)[0] * gy) + np.sum(s * gs))
    _close(gx, _differences(loss, s))
    _close(gw, _differences(loss, w))


def test_norm_by_hand():
    y, s = oracle.add_rmsnorm(np.float32([[1, 2]]), np.float32([[2, 2]]), np.array([2.0, 0.5]), 0.0)
    rms = np.sqrt((9 + 16) / 2)
    assert np.array_equal(s, [[3, 4]]) and np.allclose(y, [[6 / rms, 2 / rms]], atol=1e-15)
    # the sum is rounded to the stream's type: 2048 + 1 is not a half
    _, s = oracle.add_rmsnorm(np.float16([[2048]]), np.float16([[1]]), np.array([1.0]), 0.0)
    assert s[0, 0] == 2048


def test_e4m3_values():
    v = oracle.e4m3_values()
    assert len(v) == 127 and v[0] == 0 and v[1] == 2.0 ** -9 and v[-1] == 448 and v[-2] == 416
    assert np.all(np.diff(v) > 0) and 1.0 in v and 1.125 in v
