"""GPU: a block's token mixer in training, as its parts are used together: the
residual norm, the projections (plain products), the gated forward, and the
gradients of all of them back to the block's input and weights, against
float64 autograd through the same formulas on the CPU.

The bar is 1% of the largest gradient: every tensor between the parts is
rounded to half (2^-11 relative each, about ten of them in a row, and the
forward's own 5e-3 of the largest output on o), and rows of o near zero are
divided by their size in the gate."""
import numpy as np
import pytest
import torch

from gpu_util import say
from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def _reference(x, res, wn, proj, nw, gy, gh, gw, H, dk, dv):
    leaves = [t.double().cpu().requires_grad_() for t in (x, res, wn, *proj, nw)]
    x, res, wn, Wq, Wk, Wv, Wg, Wz, nw = leaves
    s = x + res
    h = s / (s.square().mean(-1, keepdim=True) + EPS).sqrt() * wn
    B, T, _ = h.shape
    q, k, v, z = (( h @ W).view(B, T, H, -1) for W in (Wq, Wk, Wv, Wz))
    g = torch.nn.functional.logsigmoid((h @ Wg).view(B, T, H, dk)) / 4
    order = torch.arange(T).view(gh, gw).t().reshape(-1)  # top to bottom
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64)
    rows = [None] * T
    for t in order.tolist():
        S = S * g[:, t].exp()[..., None] + k[:, t][..., None] * v[:, t][..., None, :]
        rows[t] = (q[:, t][..., None] * S).sum(2)
    o = torch.stack(rows, 1)
    y = o / (o.square().mean(-1, keepdim=True) + EPS).sqrt() * nw * torch.nn.functional.silu(z)
    loss = (y * gy.double().cpu()).sum() + s.sum()
    return y, torch.autograd.grad(loss, leaves)


def test_training_step_of_a_mixer():
    torch.manual_seed(3)
    B, gh, gw, H, dk, dv, F = 2, 7, 10, 2, 32, 64, 96
    T = gh * gw
    half = lambda *shape, s=1.0: (torch.randn(*shape, device="cuda") * s).half()
    x, res = half(B, T, F), half(B, T, F)
    wn, nw = 1 + 0.1 * torch.randn(F, device="cuda"), 1 + 0.1 * torch.randn(dv, device="cuda")
    proj = [half(F, H * d, s=F ** -0.5) for d in (dk, dk, dv, dk, dv)]
    gy = half(B, T, H, dv)
    # forward
    h, s = gla.add_rmsnorm(x, res, wn, EPS)
    heads = lambda W: (h.float() @ W.float()).half().view(B, T, H, -1)
    q, k, v, a, z = (heads(W) for W in proj)
    g = (torch.nn.functional.logsigmoid(a.float()) / 4).half()
    y = gla.fwd_gated(q, k, v, g, z, nw, EPS, gh, gw, gla.T2B)
    # backward: o again from the same inputs, then the gate's, the recurrence's and the norm's gradients
    o = gla.fwd(q, k, v, g, gh, gw, gla.T2B)
    go, gz, gnw = gla.gate_bwd(o, z, nw, EPS, gy)
    gq, gkey, gv, gg = gla.bwd(q, k, v, g, go, gh, gw, gla.T2B)
    ga = (gg.float() * torch.sigmoid(-a.float()) / 4)
    flat = lambda t: t.float().reshape(B * T, -1)
    grads = [flat(t) for t in (gq, gkey, gv, ga, gz)]
    gW = [flat(h).t() @ t for t in grads]
    gh_ = sum(t @ W.float().t() for t, W in zip(grads, proj)).half().view(B, T, F)
    gx, gwn = gla.add_rmsnorm_bwd(s, wn, EPS, gh_, gsum=torch.ones_like(s))
    torch.cuda.synchronize()
    ry, (rx, rres, rwn, *rW, rnw) = _reference(x, res, wn, proj, nw, gy, gh, gw, H, dk, dv)
    names = ["y", "x", "residual", "norm weight", "Wq", "Wk", "Wv", "Wg", "Wz", "gate norm weight"]
    for n, got, want in zip(names, [y, gx, gx, gwn, *gW, gnw], [ry, rx, rres, rwn, *rW, rnw]):
        d = (got.double().cpu() - want.detach()).abs().max().item() / want.detach().abs().max().item()
        say(f"  {n}: {d:.2e} of the largest")
        assert d <= 1e-2, n


def test_serving_a_block_token_by_token():
    """A prompt through the gated forward with its state handed back, then
    tokens one by one, against the gated forward over all of it (its bar)."""
    torch.manual_seed(4)
    B, T0, T, H, dk, dv = 3, 65, 80, 2, 64, 64
    half = lambda *shape, s=1.0: (torch.randn(*shape, device="cuda") * s).half()
    q, k, v, z = half(B, T, H, dk, s=0.125), half(B, T, H, dk), half(B, T, H, dv), half(B, T, H, dv)
    g = (torch.nn.functional.logsigmoid(torch.randn(B, T, H, dk, device="cuda")) / 16).half()
    nw = 1 + 0.1 * torch.randn(dv, device="cuda")
    whole = gla.fwd_gated(q, k, v, g, z, nw, EPS, 1, T)
    cut = lambda t: t[:, :T0].contiguous()
    pool = torch.zeros(B + 4, H, dk, dv, device="cuda")
    state = torch.empty(B, H, dk, dv, device="cuda")
    y = [gla.fwd_gated(cut(q), cut(k), cut(v), cut(g), cut(z), nw, EPS, 1, T0, s_final=state)]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(T0, T):
        one = lambda a: a[:, t].contiguous()
        y.append(gla.step_gated(one(q), one(k), one(v), one(g), one(z), nw, EPS, pool, slots)[:, None])
    torch.cuda.synchronize()
    got = torch.cat(y, 1)
    d = ((got.double() - whole.double()).abs().max() / whole.double().abs().max()).item()
    say(f"  token by token: {d:.2e} of the largest")
    assert d <= 1e-2
