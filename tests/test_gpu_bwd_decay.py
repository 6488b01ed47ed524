"""GPU: gradients of the recurrence (gla_bwd) in float where decays change
sharply: tokens that forget everything beside tokens that keep. Every pair of
tokens is held to the decay between its own two tokens (tests/pairs.py), however
deep a reset before them was.

Bounds, in units u = 2^-24 of a pair's term:
  * operands: three bf16 terms each, at most 8 * 2^-25 = 4 u over the chained
    products;
  * sums: n nonzero terms, each of three chained products: 3 n u;
  * the factor F of a pair: at most six factors, each from the exponential unit
    (one ulp, 2 u) and one product: 18 u, and 12 u for the four of every chunk
    between; or, where a sub-block's own pairs are products of the tokens'
    decays, 15 of them, 45 u;
  * its exponent: a token's decay is rounded once, sums of up to 16 of them in a
    tree of four steps: 5 u of the decay between the two tokens, times ln 2: c1 =
    3.5 u per unit of log2; and 4 u of what the sub-block's mild tokens add up to,
    at most 2, four times;
  * a factor below 2^-60 may be lost in float's or bf16's subnormals.
Plus half a step of float of the value."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from pairs import pair_bounds, pair_gradients
from recurrent_vision_token_gla_amd import gla

U = 2.0 ** -24
LN2 = np.log(2.0)
NAMES = ("gq", "gkey", "gv", "ggk", "gs0")


def make(T, dk, dv, seed, carry=True):
    """One head [T, D] of unit values in float, gates to be filled in."""
    r = np.random.default_rng(seed)
    q, k, v, go = (r.standard_normal((T, d)).astype(np.float32) for d in (dk, dk, dv, dv))
    s0, gsf = (r.standard_normal((dk, dv)).astype(np.float32) if carry else None for _ in range(2))
    return [q, k, v, None, go], s0, gsf, r


def gate(log2):
    """Natural log decay of log2 decays, in float."""
    return (np.asarray(log2) * LN2).astype(np.float32)


def compare(x, s0, gsf, c0, c1=3.5, floor=2.0 ** -60):
    """gla_bwd on one head [T, D] against the pairs."""
    T, dk = x[0].shape
    dev = to_dev(*[a.reshape(1, T, 1, -1) for a in x])
    ds0, dgs = (None if a is None else to_dev(a.reshape(1, 1, dk, -1))[0] for a in (s0, gsf))
    got = gla.bwd(*dev, 1, T, 0, s0=ds0, gs_final=dgs, return_gs0=True)
    torch.cuda.synchronize()
    want = pair_gradients(x, s0, gsf)
    tol = pair_bounds(x, s0, gsf, c0 * U, c1 * U, floor)
    bad = []
    for name, a, w, t in zip(NAMES, got, want, tol):
        a = a.double().cpu().numpy().reshape(w.shape)
        worst = float(np.max(np.abs(a - w) / (t + U * np.abs(w) + 1e-36)))
        say(f"  {name}: {worst:.3f} of the bound")
        bad += [name] if not worst <= 1 else []
    assert not bad


def test_pairs_agree_with_the_recurrence():
    """CPU: the sums over pairs against the token-by-token oracle."""
    x, s0, gsf, r = make(37, 5, 4, 1)
    x[3] = gate(-np.exp(r.uniform(-5, 3, (37, 5))))
    b = lambda a: a.reshape(1, 37, 1, -1)
    want = oracle.gla_backward(*[b(a) for a in x], 1, 37, [0], s0.reshape(1, 1, 5, 4), gsf.reshape(1, 1, 5, 4))
    for a, w in zip(pair_gradients(x, s0, gsf), want):
        assert np.allclose(a, w.reshape(a.shape), rtol=1e-9, atol=1e-12)
    exact = pair_bounds(x, s0, gsf, 1.0, 0.0, 0.0)  # at least the magnitudes
    for a, e in zip(pair_gradients(x, s0, gsf), exact):
        assert np.all(np.abs(a) <= e * (1 + 1e-12))


def resets(T, dk, r, first=True):
    """Mild decays, and in three sub-blocks of four one to twelve of the first
    twelve tokens that forget everything, dim by dim."""
    g = -r.uniform(0.005, 0.06, (T, dk))
    for m in range(T // 16):
        if m % 4:
            n = r.integers(1, 13, dk)
            for d in range(dk):
                g[16 * m + r.permutation(12)[:n[d]], d] = -400.0
    return gate(g)


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", [(32, 64), (64, 64)])
def test_single_pairs_behind_resets(dk, dv):
    """One key and one query per sub-block, behind its resets, and one value
    column: sums of at most nine terms, so that the decay between the two tokens
    is what is measured. No sub-block without a reset decays by more than 2: its
    exponents add at most 4 * 2 * 4 ln 2 = 23 u."""
    T = 144
    say(f"resets, single pairs {dk}/{dv}")
    x, _, _, r = make(T, dk, dv, 11, carry=False)
    x[3] = resets(T, dk, r)
    for i, at in ((0, 15), (1, 13), (2, 13), (4, 15)):
        keep = x[i][at::16].copy()
        x[i][:] = 0
        x[i][at::16] = keep
    x[2][:, 1:] = 0
    x[4][:, 1:] = 0
    compare(x, None, None, 4 + 3 * 9 + 45 + 23 + 12 * 3)



@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64)])
def test_dense_values_among_resets(dk, dv):
    """All tokens, a carried state and a gradient of the final one: sums of up to
    dv products and 64 tokens and three chunks' states."""
    T = 144
    say(f"resets, dense {dk}/{dv}")
    x, s0, gsf, r = make(T, dk, dv, 12)
    x[3] = resets(T, dk, r)
    compare(x, s0, gsf, 4 + 3 * 64 + 3 + 45 + 23 + 12 * 3)



@pytest.mark.gpu
def test_chunks_between_resets():
    """Resets every 50 tokens over five chunks: what passes from chunk to chunk is
    exact to the decay between the tokens."""
    T = 320
    x, s0, gsf, r = make(T, 32, 32, 16)
    g = -r.uniform(0.005, 0.03, (T, 32))
    g[::50] = -300.0
    x[3] = gate(g)
    say("resets every 50 tokens")
    compare(x, s0, gsf, 4 + 3 * 64 + 5 + 45 + 23 + 12 * 5)
