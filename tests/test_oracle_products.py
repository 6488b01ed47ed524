"""The oracle of the products and norms between a block's mixers against values
worked out by hand, torch's float64 functions and autograd, and central
differences (CPU).

Against torch both sides are float64 sums of at most 40 terms of order one: the
bar is 1e-12 of the largest value. A central difference with h = 1e-4 of values
of order one is off by about 1e-8: the bar is 1e-6 of the largest gradient."""
import math

import numpy as np
import pytest
import torch

import oracle

KINDS = ["none", "silu", "gelu", "logsigmoid"]
F = torch.nn.functional
TORCH = {"none": lambda z: z, "silu": F.silu, "gelu": F.gelu, "logsigmoid": F.logsigmoid}
EPS = 1e-6


def close(got, want, bar=1e-12):
    want = want.detach().numpy() if torch.is_tensor(want) else want
    assert np.max(np.abs(got - want)) <= bar * max(1.0, np.max(np.abs(want)))


def leaf(a):
    return None if a is None else torch.from_numpy(np.asarray(a, dtype=np.float64)).requires_grad_()


def test_activations_at_known_points():
    assert oracle.act(0.0, "silu") == 0 and oracle.act(0.0, "gelu") == 0
    assert abs(oracle.act(0.0, "logsigmoid") + math.log(2)) < 1e-15
    assert abs(oracle.act(1.0, "silu") - 1 / (1 + math.exp(-1))) < 1e-15
    assert abs(oracle.act(1.0, "gelu") - 0.8413447460685429) < 1e-14  # Phi(1)
    assert abs(oracle.act(-40.0, "logsigmoid") + 40) < 1e-14
    assert oracle.act(-30.0, "gelu") < 0  # the lower tail is not lost
    assert oracle.act(3.5, "none") == 3.5 and oracle.act_slope(3.5, "none") == 1


@pytest.mark.parametrize("kind", KINDS)
def test_activations_match_torch(kind):
    z = np.linspace(-12, 12, 241)
    t = leaf(z)
    y = TORCH[kind](t)
    close(oracle.act(z, kind), y)
    close(oracle.act_slope(z, kind), torch.autograd.grad(y.sum(), t)[0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("with_bias", [True, False])
def test_linear_and_gradient(kind, with_bias):
    r = np.random.default_rng(5)
    x, w, b, res, gy = (r.standard_normal(s) for s in ((7, 40), (24, 40), (24,), (7, 24), (7, 24)))
    if not with_bias:
        b = None
    tx, tw, tb = leaf(x), leaf(w), leaf(b)
    y = 0.125 * TORCH[kind](F.linear(tx, tw, tb)) + torch.from_numpy(res)
    got, pre = oracle.linear(x, w, b, kind, 0.125, res)
    close(got, y)
    close(pre, F.linear(tx, tw, tb))
    leaves = [t for t in (tx, tw, tb) if t is not None]
    for g, want in zip(oracle.linear_backward(x, w, pre, gy, kind, 0.125),
                       torch.autograd.grad((y * torch.from_numpy(gy)).sum(), leaves)):
        close(g, want)


@pytest.mark.parametrize("kind", KINDS)
def test_gated_ff_and_gradient(kind):
    r = np.random.default_rng(6)
    x, wg, wu, gh = (r.standard_normal(s) for s in ((5, 24), (16, 24), (16, 24), (5, 16)))
    leaves = [leaf(t) for t in (x, wg, wu)]
    h = TORCH[kind](F.linear(leaves[0], leaves[1])) * F.linear(leaves[0], leaves[2])
    got, a, u = oracle.gated_ff(x, wg, wu, kind)
    close(got, h)
    for g, want in zip(oracle.gated_ff_backward(x, wg, wu, a, u, gh, kind),
                       torch.autograd.grad((h * torch.from_numpy(gh)).sum(), leaves)):
        close(g, want)


@pytest.mark.parametrize("post,gated,scaled,groups", [(1, 1, 1, 3), (1, 0, 1, 1), (0, 1, 0, 6), (0, 0, 0, 1), (1, 1, 0, 1)])
def test_gated_add_rmsnorm_and_gradient(post, gated, scaled, groups):
    r = np.random.default_rng(7)
    rows, width = 6, 16
    x, res, gy, gs = (r.standard_normal((rows, width)) for _ in range(4))
    w, b, f = (1 + 0.2 * r.standard_normal(width) for _ in range(3))
    g = r.standard_normal((groups, width))
    b, g, f = b if post else None, g if gated else None, f if scaled else None
    tx, tr, tw, tb, tg, tf = map(leaf, (x, res, w, b, g, f))
    p = tx if tb is None else F.rms_norm(tx, (width,), tb, EPS)
    if tg is not None:
        p = p * tg.repeat_interleave(rows // groups, 0)
    s = tr + (p if tf is None else p * tf)
    y = F.rms_norm(s, (width,), tw, EPS)
    got, gots, whole = oracle.gated_add_rmsnorm(x, res, w, EPS, b, g, f)
    close(got, y)
    close(gots, s)
    assert np.array_equal(gots, whole)  # float64 rows are not rounded
    names = [("x", tx), ("residual", tr), ("weight", tw), ("post", tb), ("gate", tg), ("scale", tf)]
    grads = oracle.gated_add_rmsnorm_backward(x, gots, w, EPS, gy, gs, b, g, f)
    want = torch.autograd.grad((y * torch.from_numpy(gy)).sum() + (s * torch.from_numpy(gs)).sum(),
                               [t for _, t in names if t is not None])
    want = iter(want)
    for (name, t), got in zip(names, grads):
        if t is None:
            assert got is None, name
        else:
            close(got, next(want))


def test_rounded_sum_is_what_the_norm_is_of():
    x = np.array([[1.0, 0, 0, 0, 0, 0, 0, 0]], np.float16)
    res = np.full((1, 8), 2.0 ** -12, np.float16)
    y, s, whole = oracle.gated_add_rmsnorm(x, res, np.ones(8), 0.0)
    assert whole[0, 0] == 1 + 2.0 ** -12 and s[0, 0] == 1.0
    assert abs(y[0, 0] - 1 / math.sqrt((1 + 7 * 2.0 ** -24) / 8)) < 1e-12


def test_gradients_match_differences():
    r = np.random.default_rng(8)
    x, res, gy, gs = (r.standard_normal((4, 8)) for _ in range(4))
    w, b, f = (1 + 0.2 * r.standard_normal(8) for _ in range(3))
    g = r.standard_normal((2, 8))
    _, s, _ = oracle.gated_add_rmsnorm(x, res, w, EPS, b, g, f)
    grads = oracle.gated_add_rmsnorm_backward(x, s, w, EPS, gy, gs, b, g, f)

    def loss():
        y, s, _ = oracle.gated_add_rmsnorm(x, res, w, EPS, b, g, f)
        return float((y * gy).sum() + (s * gs).sum())

    for t, got in zip((x, res, w, b, g, f), grads):
        want = np.zeros_like(t)
        for i in np.ndindex(*t.shape):
            keep, v = t[i], []
            for h in (1e-4, -1e-4):
                t[i] = keep + h
                v.append(loss())
            t[i] = keep
            want[i] = (v[0] - v[1]) / 2e-4
        close(got, want, 1e-6)


def test_planted_mistakes_are_caught(monkeypatch):
    """Each slip makes at least one check above fail."""
    import oracle.products as P
    slips = [("act", lambda z, k, f=P.act: f(z, "silu" if k == "gelu" else k)),
             ("act_slope", lambda z, k, f=P.act_slope: f(-np.asarray(z, float), k)),
             ("_per_row", lambda g, n: np.ones((1, 1)) if g is None else np.tile(g, (n // len(g), 1))),
             ("_rstd", lambda s, e: 1 / np.sqrt(np.sum(s * s, -1, keepdims=True) + e))]
    for name, wrong in slips:
        with monkeypatch.context() as m:
            m.setattr(P, name, wrong)
            if hasattr(oracle, name):
                m.setattr(oracle, name, wrong)
            with pytest.raises(AssertionError):
                for k in KINDS:
                    test_activations_match_torch(k)
                    test_linear_and_gradient(k, True)
                test_gated_add_rmsnorm_and_gradient(1, 1, 1, 3)
