"""Float64 oracle of the products and norms between a block's mixers and of
their gradients. TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

    linear      y = alpha act(x W^T + b) + residual
    gated_ff    h = act(x Wg^T) * (x Wu^T)
    gated_add_rmsnorm
                p = x / rms(x) * post, s = residual + scale gate p rounded to
                x's dtype, y = s / rms(s) * w, with one gate row for each of
                equal groups of rows

Activations are named: none, silu z / (1 + exp(-z)), gelu z Phi(z),
logsigmoid -log(1 + exp(-z))."""
from __future__ import annotations

import numpy as np
from scipy.special import erfc


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def _sigmoid(z):
    return np.exp(-np.logaddexp(0.0, -z))


def act(z, kind: str) -> np.ndarray:
    z = _f64(z)
    if kind == "silu":
        return z * _sigmoid(z)
    if kind == "gelu":
        return z * erfc(-z / np.sqrt(2.0)) / 2.0
    if kind == "logsigmoid":
        return -np.logaddexp(0.0, -z)
    return z


def act_slope(z, kind: str) -> np.ndarray:
    z = _f64(z)
    if kind == "silu":
        s = _sigmoid(z)
        return s + z * s * (1.0 - s)
    if kind == "gelu":
        return erfc(-z / np.sqrt(2.0)) / 2.0 + z * np.exp(-z * z / 2.0) / np.sqrt(2.0 * np.pi)
    if kind == "logsigmoid":
        return _sigmoid(-z)
    return np.ones_like(z)


def linear(x, weight, bias=None, kind="none", alpha=1.0, residual=None):
    """(y, pre) for rows x [rows, K], weight [N, K]."""
    pre = _f64(x) @ _f64(weight).T
    if bias is not None:
        pre = pre + _f64(bias)
    y = float(alpha) * act(pre, kind)
    return (y if residual is None else y + _f64(residual)), pre


def linear_backward(x, weight, pre, gy, kind="none", alpha=1.0):
    """(gx, gweight, gbias) from the kept pre (None without activation)."""
    gp = float(alpha) * _f64(gy)
    if kind != "none":
        gp = gp * act_slope(pre, kind)
    return gp @ _f64(weight), gp.T @ _f64(x), gp.sum(0)


def gated_ff(x, gate_weight, up_weight, kind="silu"):
    """(h, a, u)."""
    a, u = _f64(x) @ _f64(gate_weight).T, _f64(x) @ _f64(up_weight).T
    return act(a, kind) * u, a, u


def gated_ff_backward(x, gate_weight, up_weight, a, u, gh, kind="silu"):
    """(gx, ggate_weight, gup_weight)."""
    x, a, u, gh = map(_f64, (x, a, u, gh))
    ga, gu = gh * u * act_slope(a, kind), gh * act(a, kind)
    return ga @ _f64(gate_weight) + gu @ _f64(up_weight), ga.T @ x, gu.T @ x


def _rstd(s, eps):
    return 1.0 / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + float(eps))


def _per_row(gate, rows):
    return np.ones((1, 1)) if gate is None else np.repeat(_f64(gate), rows // len(gate), axis=0)


def gated_add_rmsnorm(x, residual, weight, eps, post=None, gate=None, scale=None):
    """(y, s, exact s) for rows x [rows, F], gate [groups, F]: y of the rounded s."""
    m = _f64(x)
    p = m if post is None else m * _rstd(m, eps) * _f64(post)
    f = 1.0 if scale is None else _f64(scale)
    whole = _f64(residual) + f * _per_row(gate, len(m)) * p
    s = _f64(whole.astype(np.asarray(x).dtype))
    return s * _rstd(s, eps) * _f64(weight), s, whole


def gated_add_rmsnorm_backward(x, s, weight, eps, gy, gsum=None, post=None, gate=None, scale=None):
    """(gx, gresidual, gweight, gpost, ggate, gscale), None for those without
    an input."""
    m, s, gy, w = map(_f64, (x, s, gy, weight))
    rs = _rstd(s, eps)
    n = s * rs
    gS = rs * (gy * w - n * np.mean(gy * w * n, axis=-1, keepdims=True))
    if gsum is not None:
        gS = gS + _f64(gsum)
    g = _per_row(gate, len(m))
    f = np.ones(m.shape[-1]) if scale is None else _f64(scale)
    b = np.ones(m.shape[-1]) if post is None else _f64(post)
    nx = m if post is None else m * _rstd(m, eps)
    gn = gS * f * g * b
    gx = gn if post is None else _rstd(m, eps) * (gn - nx * np.mean(gn * nx, axis=-1, keepdims=True))
    ggate = None
    if gate is not None:
        ggate = (gS * f * b * nx).reshape(len(gate), -1, m.shape[-1]).sum(1)
    return (gx, gS, (gy * n).sum(0), None if post is None else (gS * f * g * nx).sum(0), ggate,
            None if scale is None else (gS * g * b * nx).sum(0))
