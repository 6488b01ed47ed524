"""The recurrence's gradient in float64 as sums over pairs of tokens, and what
each output may be off by if every pair is held to the decay between its own
two tokens. TEST INFRASTRUCTURE.

For one (batch, head) in scan order, with b the inclusive cumulative log2 decay
and F_ij = 2^(b_i - b_j), j <= i, P_ij = go_i . v_j:
  gq_i  = sum_j P_ij k_j F_ij + 2^b_i S0 go_i
  gk_j  = sum_i P_ij q_i F_ij + 2^(b_T - b_j) G v_j
  gv_j  = sum_i (sum_d q_i k_j F_ij) go_i + G^T (k_j 2^(b_T - b_j))
  gg_t  = sum_{i >= t > j} P_ij q_i k_j F_ij + sum_{i >= t} q_i 2^b_i S0 go_i
        + sum_{j < t} k_j 2^(b_T - b_j) G v_j + 2^b_T <S0, G>
  gs0   = sum_i 2^b_i q_i^T go_i + 2^b_T G
"""
import numpy as np

MIN_LOG2 = -160.0  # a token's decay counts as at least this


def pair_gradients(x, s0, gsf, weigh=None):
    """Gradients (gq, gk, gv, gg, gs0) of one head, inputs [T, D]. With weigh(D),
    D = b_i - b_j <= 0, every term is taken in magnitude and times it."""
    q, k, v, g, go = (a.astype(np.float64) for a in x)
    T, dk = q.shape
    s0 = np.zeros((dk, v.shape[1])) if s0 is None else s0.astype(np.float64)
    gsf = np.zeros_like(s0) if gsf is None else gsf.astype(np.float64)
    b = np.cumsum(np.maximum(g * np.log2(np.e), MIN_LOG2), 0)
    f = lambda d: np.exp2(d) * (1.0 if weigh is None else weigh(d))
    if weigh is not None:
        q, k, v, go, s0, gsf = (np.abs(a) for a in (q, k, v, go, s0, gsf))
    causal = np.tril(np.ones((T, T), bool))
    F = np.where(causal[..., None], f(np.where(causal[..., None], b[:, None] - b[None], 0.0)), 0.0)
    start, end, whole = f(b), f(b[-1] - b), f(b[-1])  # from before the first token, to the end
    P = go @ v.T
    from_s, from_g = start * (go @ s0.T), end * (v @ gsf.T)
    gq = np.einsum("ij,jd,ijd->id", P, k, F) + from_s
    gk = np.einsum("ij,id,ijd->jd", P, q, F) + from_g
    A = np.einsum("id,jd,ijd->ij", q, k, F)
    gv = A.T @ go + (k * end) @ gsf
    W = P[..., None] * q[:, None] * k[None] * F
    W[np.arange(T), np.arange(T)] = 0
    cross = np.empty_like(q)
    for t in range(T):  # pairs i >= t > j
        cross[t] = W[t:, :t].sum((0, 1))
    before = np.cumsum(k * from_g, 0) - k * from_g
    gg = cross + np.cumsum((q * from_s)[::-1], 0)[::-1] + before + whole * (s0 * gsf).sum(1)
    gs0 = (q * start).T @ go + whole[:, None] * gsf
    return gq, gk, gv, gg, gs0


def pair_bounds(x, s0, gsf, c0, c1, floor, chunk=64):
    """What the outputs may be off by where a pair's term may be off by
    c0 + c1 |b_i - b_j| of itself, or by `floor` of what it is without decay.
    The decay's gradient takes differences inside a chunk: it adds twice the
    sum of |q gq| over the chunk's tokens behind."""
    off = list(pair_gradients(x, s0, gsf, lambda d: c0 - c1 * d + floor * np.exp2(np.minimum(-d, 1000.0))))
    T = len(off[0])
    z = np.abs(x[0].astype(np.float64)) * off[0]
    for n in range(0, T, chunk):
        off[3][n:n + chunk] += 2 * np.cumsum(z[n:n + chunk][::-1], 0)[::-1]
    return off
