"""GPU: gradients of the recurrence (gla_bwd) in float where decays change
sharply: tokens that forget everything beside tokens that keep, and sub-blocks
of 16 tokens near the largest decay that shares one reference. Every pair of
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
    3.5 u per unit of log2; where a sub-block has a reference, two tokens'
    distances to it, at most 66 each, with 4 u each: 4 * 66 * 2 ln 2 = 366 u, and
    for two sub-blocks the references' distances to the blocks' ends as well: 735 u;
  * a factor below 2^-60 may be lost in float's or bf16's subnormals: floor 2^-62
    where only sums in float pass through them, 2^-60 otherwise.
Plus half a step of the output's type of the value."""
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
        step = 2.0 ** -11 * np.abs(w) + 2.0 ** -25 if a.dtype == torch.float16 else U * np.abs(w) + 1e-36
        a = a.double().cpu().numpy().reshape(w.shape)
        worst = float(np.max(np.abs(a - w) / (t + step)))
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
@pytest.mark.parametrize("deep", [-20.0, -55.0, -90.0, -400.0])
@pytest.mark.parametrize("token", [0, 7, 8])
def test_single_pairs_behind_one_reset(token, deep):
    """The same with one reset per sub-block in all dims, of any depth: at its
    first token (rows of a grid that forget the row before), and beside its
    middle. Two tokens on one side of it have distances to the reference that
    hold it both, 366 u, or none."""
    T = 144
    say(f"one reset of 2^{deep} at token {token}")
    x, _, _, r = make(T, 32, 32, 17, carry=False)
    g = -r.uniform(0.005, 0.06, (T, 32))
    g[token::16] = deep
    x[3] = gate(g)
    for i, at in ((0, 15), (1, 13), (2, 13), (4, 15)):
        keep = x[i][at::16].copy()
        x[i][:] = 0
        x[i][at::16] = keep
    x[2][:, 1:] = 0
    x[4][:, 1:] = 0
    compare(x, None, None, 4 + 3 * 9 + 45 + 23 + 12 * 3 + (366 if deep > -66 and token > 7 else 0))


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
@pytest.mark.parametrize("log2", [-2.0, -5.0, -7.2, -8.24, -8.26, -8.49, -8.51, -9.0, -12.0, -30.0])
def test_constant_decays(log2):
    """Every token decays alike, around the largest decay with a reference (66
    over eight tokens)."""
    say(f"constant 2^{log2}")
    x, s0, gsf, r = make(100, 64, 32, 13)
    x[3] = gate(np.full((100, 64), log2))
    compare(x, s0, gsf, 4 + 3 * 64 + 2 + 45 + 735 + 12 * 2)


@pytest.mark.gpu
@pytest.mark.parametrize("deep", [7.9, 8.5, 9.3])
@pytest.mark.parametrize("between", [0, 1, 2])
def test_pairs_between_two_strong_stretches(deep, between):
    """Seven strong tokens at the end of one sub-block but its last, and seven
    after the first token of a later one: the tokens next to them keep each
    other through one or two sub-blocks that decay by 2^-14 each, however small
    the factor between the two blocks' references is."""
    say(f"strong stretches of 7 x 2^-{deep}, {between} sub-blocks between")
    T = 80
    x, s0, gsf, r = make(T, 32, 32, 14)
    g = np.full((T, 32), -0.01)
    g[8:15] = -deep
    g[16:16 * (between + 1)] = -14 / 16
    i = 16 * (between + 1)
    g[i + 1:i + 8] = -deep
    x[3] = gate(g)
    for a in (x[1], x[2]):
        a[np.arange(T) != 15] = 0
    for a in (x[0], x[4]):
        a[np.arange(T) != i] = 0
    compare(x, None, None, 4 + 3 * 32 + 45 + 735)


@pytest.mark.gpu
def test_state_behind_a_reset_and_strong_tokens():
    """A sub-block whose first token decays by 2^-58 and the next seven to 2^-126:
    what its first query takes from the entering state is 2^-58 of it, and there
    is no key whose own pair would hide that."""
    say("state behind a reset and strong tokens")
    x, s0, gsf, r = make(32, 32, 32, 15)
    g = np.full((32, 32), -0.01)
    g[0] = -58.5
    g[1:8] = -68.0 / 7
    x[3] = gate(g)
    x[1][:] = 0
    x[0][1:] = 0
    x[4][1:] = 0
    compare(x, s0, None, 4 + 3 * 32 + 45 + 735, floor=2.0 ** -62)


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


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(16))
def test_random_decays(seed):
    """Each sub-block of its own kind: mild, constant by dim, from weak to strong,
    deep tokens in some dims, tokens that forget everything, just at the largest
    distance with a reference. Half inputs add the 512 u of two-term operands
    (8 * 2^-18) and half a step of their type."""
    r = np.random.default_rng(1900 + seed)
    T, half, carry = int(r.integers(1, 200)), bool(seed % 2), bool(r.integers(2))
    dk, dv = (int(r.choice([32, 64])) for _ in range(2))
    say(f"random decays seed={seed} T={T} {dk}/{dv} half={half} carry={carry}")
    x, s0, gsf, _ = make(T, dk, dv, 1950 + seed, carry=carry)
    g = np.zeros((T, dk))
    for m in range(0, T, 16):
        s = g[m:m + 16].shape
        g[m:m + 16] = [lambda: -r.uniform(0, 0.1, s), lambda: -r.uniform(0, 9, (1, dk)),
                       lambda: -np.exp(r.uniform(-8, 5, s)),
                       lambda: np.where(r.random(s) < 0.1, -r.uniform(20, 70), -0.02),
                       lambda: np.where(r.random((s[0], 1)) < 0.1, -8e4, -0.02),
                       lambda: -r.uniform(6, 9.4)][int(r.integers(6))]()
    x[3] = gate(g)
    if half:
        x = [a.astype(np.float16) for a in x]
    compare(x, s0, gsf, 4 + 3 * 64 + 45 + 735 + 12 * 4 + (512 if half else 0))


@pytest.mark.gpu
@pytest.mark.parametrize("reset", [False, True])
def test_nan_reaches_only_the_pairs_that_have_it(reset):
    """A NaN in one token's v, and in another's go, inside one sub-block, with and
    without a token that forgets everything: queries before the first and keys
    behind the second do not meet them."""
    say(f"NaN inside a sub-block, reset={reset}")
    x, _, _, r = make(16, 32, 32, 18, carry=False)
    g = -r.uniform(0.005, 0.06, (16, 32))
    if reset:
        g[7] = -400.0
    x[3] = gate(g)
    dev = to_dev(*[a.reshape(1, 16, 1, -1) for a in x])
    clean = gla.bwd(*dev, 1, 16, 0)
    v, go = dev[2].clone(), dev[4].clone()
    v[0, 10, 0, 3] = go[0, 4, 0, 5] = float("nan")
    got_v = gla.bwd(dev[0], dev[1], v, dev[3], dev[4], 1, 16, 0)
    got_go = gla.bwd(*dev[:4], go, 1, 16, 0)
    torch.cuda.synchronize()
    keep = [t for t in range(16) if t != 10]
    assert torch.equal(got_v[0][0, :10], clean[0][0, :10]) and bool(got_v[0][0, 10:].isnan().all())
    assert torch.equal(got_v[1][0, keep], clean[1][0, keep]) and torch.equal(got_v[2], clean[2])
    assert torch.equal(got_go[1][0, 5:], clean[1][0, 5:]) and bool(got_go[1][0, :5].isnan().all())
    keep = [t for t in range(16) if t != 4]
    assert torch.equal(got_go[0][0, keep], clean[0][0, keep])
