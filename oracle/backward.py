"""Float64 oracle of the gradients, the residual norm and its 8-bit output.
TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Gradient of the recurrence S_t = diag(exp(g_t)) S_{t-1} + k_t^T v_t,
o_t = q_t S_t (GTR project page, "How GTR Works") by the chain rule, token by
token: with E_t the gradient of S_t,

    E_t = diag(exp(g_{t+1})) E_{t+1} + q_t^T go_t   (E after the end: gs_final)
    gq_t = S_t go_t, gk_t = E_t v_t, gv_t = E_t^T k_t,
    gg_t[d] = sum_e exp(g_t[d]) S_{t-1}[d, e] E_t[d, e],  gs0 = diag(exp(g_1)) E_1.

The norms follow oracle.rmsnorm_gate's formula (ai.info summary of GTR,
"Methodology in Plain English") and its derivative.
"""
from __future__ import annotations

from typing import Sequence

import numpy as np

from .epilogue import silu
from .scan_order import to_raster, to_scan


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def recurrence_backward(q, k, v, g, go, s0=None, gs_final=None, segment: int = 64):
    """Scan-ordered [B, T, H, D] inputs -> (gq, gk, gv, gg, gs0) in float64.
    The states are kept at every `segment` tokens and computed again between."""
    q, k, v, g, go = map(_f64, (q, k, v, g, go))
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    step = lambda S, t: np.exp(g[:, t])[..., None] * S + k[:, t][..., None] * v[:, t][:, :, None, :]
    S = np.zeros((B, H, dk, dv)) if s0 is None else _f64(s0).copy()
    kept = []
    for t in range(T):
        if t % segment == 0:
            kept.append(S)
        S = step(S, t)
    E = np.zeros((B, H, dk, dv)) if gs_final is None else _f64(gs_final).copy()  # behind token t
    gq, gk, gv, gg = (np.zeros_like(x) for x in (q, k, v, g))
    for n in range(len(kept) - 1, -1, -1):
        states = [kept[n]]  # before each token of the segment, and behind the last
        for t in range(n * segment, min(T, (n + 1) * segment)):
            states.append(step(states[-1], t))
        for t in range(min(T, (n + 1) * segment) - 1, n * segment - 1, -1):
            E = E + q[:, t][..., None] * go[:, t][:, :, None, :]
            before, after = states[t - n * segment], states[t - n * segment + 1]
            gq[:, t] = np.einsum("bhde,bhe->bhd", after, go[:, t])
            gk[:, t] = np.einsum("bhde,bhe->bhd", E, v[:, t])
            gv[:, t] = np.einsum("bhde,bhd->bhe", E, k[:, t])
            E_in = np.exp(g[:, t])[..., None] * E
            gg[:, t] = np.einsum("bhde,bhde->bhd", before, E_in)
            E = E_in
    return gq, gk, gv, gg, E


def gla_backward(q, k, v, gk, go, grid_h: int, grid_w: int, dirs: Sequence[int], s0=None,
                 gs_final=None):
    """Raster-ordered [B, T, H, D] inputs -> raster-ordered gradients of q, k,
    v, gk and the gradient of s0, in float64 (states carry no spatial order)."""
    s = lambda x: to_scan(_f64(x), grid_h, grid_w, dirs)
    *grads, gs0 = recurrence_backward(s(q), s(k), s(v), s(gk), s(go), s0, gs_final)
    return tuple(to_raster(x, grid_h, grid_w, dirs) for x in grads) + (gs0,)


def rmsnorm_gate_backward(o, gate, weight, eps: float, gy):
    """(go, ggate, gweight) of rmsnorm_gate for rows [..., dv]."""
    o, z, w, gy = map(_f64, (o, gate, weight, gy))
    rstd = 1.0 / np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + float(eps))
    n, sig = o * rstd, 1.0 / (1.0 + np.exp(-z))
    gn = gy * w * silu(z)
    go = rstd * (gn - n * np.mean(gn * n, axis=-1, keepdims=True))
    gz = gy * n * w * (sig + z * sig * (1.0 - sig))
    return go, gz, np.sum((gy * n * silu(z)).reshape(-1, o.shape[-1]), axis=0)


def add_rmsnorm(x, residual, weight, eps: float):
    """(y, s): s = x + residual rounded to x's dtype, y = RMSNorm(s) * weight."""
    s = _f64(x) if residual is None else _f64((_f64(x) + _f64(residual)).astype(np.asarray(x).dtype))
    return s / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + float(eps)) * _f64(weight), s


def add_rmsnorm_backward(s, weight, eps: float, gy, gsum=None):
    """(gx, gweight) of add_rmsnorm from its s."""
    s, w, gy = map(_f64, (s, weight, gy))
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + float(eps))
    n, gn = s * rstd, gy * w
    gx = rstd * (gn - n * np.mean(gn * n, axis=-1, keepdims=True))
    if gsum is not None:
        gx = gx + _f64(gsum)
    return gx, np.sum((gy * n).reshape(-1, s.shape[-1]), axis=0)


def e4m3_values() -> np.ndarray:
    """The non-negative finite values of OCP e4m3, ascending: 4 exponent bits
    (bias 7), 3 mantissa bits, 448 the largest."""
    sub = np.arange(8) / 8.0 * 2.0 ** -6
    normal = [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.concatenate([sub, np.array(normal[:-1])])  # the last code is NaN
