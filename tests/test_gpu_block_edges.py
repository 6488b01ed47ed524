"""GPU: the products and norms between a block's mixers at the edges of what they
take: empty batches, sums and gradients beyond half's range on their way.

Tolerances are those of test_gpu_linear.py; half values that were divided by 2^p
before they were rounded are off by 2^(p - 25) below the smallest normal."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla
from test_gpu_linear import ACTS, U, act_off, check, half_step, normal, sums

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def test_no_images_and_a_gate_of_each():
    """An empty batch has no row of a gate with one row for each image either."""
    w = torch.ones(64, device="cuda")
    for lead in ((0, 5), (0,)):
        x = torch.empty(*lead, 64, device="cuda").half()
        gate = torch.empty(0, 64, device="cuda").half()
        y, s = gla.gated_add_rmsnorm(x, x, w, EPS, gate=gate, scale=w)
        gx, gres, gw, gpost, ggate, gscale = gla.gated_add_rmsnorm_bwd(x, s, w, EPS, y, gate=gate, scale=w)
        torch.cuda.synchronize()
        assert y.shape == s.shape == gx.shape == gres.shape == x.shape and ggate.shape == gate.shape
        assert gpost is None and not gw.any() and not gscale.any()
    rows = torch.randn(3, 64, device="cuda").half()
    with pytest.raises(ValueError):  # rows without a gate of theirs
        gla.gated_add_rmsnorm(rows, rows, w, EPS, gate=rows[:0])


def large_gated(rows, K, F, kind, seed):
    """Inputs whose ga and gu pass 65504 on the way to gradients that do not."""
    r = np.random.default_rng(seed)
    x = normal(r, np.float16, rows, K, s=2.0 ** -10)
    wg, wu = (normal(r, np.float16, F, K, s=2.0 ** -11) for _ in range(2))
    a, u = normal(r, np.float16, rows, F, s=3.0), normal(r, np.float16, rows, F, s=300.0)
    gh = normal(r, np.float16, rows, F, s=200.0)
    gh[0, 0], u[0, 0], a[0, 0] = 300, 1000, 2
    return x, wg, wu, a, u, gh


# one tile, both products in one launch and in two, the weights' rows split
@pytest.mark.parametrize("rows,K,F", [(1, 8, 8), (3, 72, 24), (65, 64, 64), (700, 72, 136), (2100, 264, 520),
                                      (5000, 520, 1032)])
@pytest.mark.parametrize("kind", ["silu", "gelu", "none"])
def test_gated_gradient_beyond_halfs_range_on_the_way(rows, K, F, kind):
    x, wg, wu, a, u, gh = large_gated(rows, K, F, kind, rows + K + F + 4)
    got = gla.gated_ff_bwd(*to_dev(x, wg, wu, a, u, gh), act=ACTS[kind])
    torch.cuda.synchronize()
    say(f"gated_ff_bwd {rows}x{K}x{F} {kind}, large")
    want = oracle.gated_ff_backward(x, wg, wu, a, u, gh, kind)
    z, v, g = (t.astype(np.float64) for t in (a, u, gh))
    ga, gu = g * v * oracle.act_slope(z, kind), g * oracle.act(z, kind)
    most = max(np.abs(ga).max(), np.abs(gu).max())
    assert most > 65520 and all(np.abs(w).max() < 60000 for w in want)
    step = lambda t: 2.0 ** -11 * np.abs(t) + 2.0 ** (np.floor(np.log2(most)) - 14 - 25)
    off = 0 * z if kind == "none" else act_off(z)
    oa, ou = off * 1.13 * np.abs(g * v) + 4 * U * np.abs(ga) + step(ga), off * np.abs(gu) + 4 * U * np.abs(gu) + step(gu)
    A, B, X = np.abs(ga) + oa, np.abs(gu) + ou, np.abs(x.astype(np.float64))
    Wg, Wu = (np.abs(w.astype(np.float64)) for w in (wg, wu))
    check("gx", got[0], want[0], oa @ Wg + ou @ Wu + sums(np.float16, 2 * F, A @ Wg + B @ Wu) +
          half_step(np.float16, want[0]))
    for name, k, o, t in (("ggate_weight", 1, oa, A), ("gup_weight", 2, ou, B)):
        check(name, got[k], want[k], o.T @ X + sums(np.float16, rows, t.T @ X) + half_step(np.float16, want[k]))


def test_large_gated_gradient_beside_infinities_and_in_a_graph():
    """What is not finite does not count as the largest, and stays in its rows of
    gx; a captured call takes the scale of the inputs it is replayed with."""
    inputs = [to_dev(*large_gated(300, 72, 136, "silu", seed)) for seed in (1, 2)]
    small = [t.clone() for t in inputs[0]]
    small[5] /= 256
    clean = gla.gated_ff_bwd(*inputs[0])
    bad = [t.clone() for t in inputs[0]]
    bad[5][7, 3], bad[4][9, 5], bad[3][11, 1] = float("nan"), float("inf"), float("nan")
    got = gla.gated_ff_bwd(*bad)
    torch.cuda.synchronize()
    keep = [i for i in range(300) if i not in (7, 9, 11)]
    assert torch.equal(got[0][keep], clean[0][keep]) and all(torch.isfinite(t).all() for t in clean)
    assert not torch.isfinite(got[0][[7, 9, 11]]).any()
    static = [t.clone() for t in inputs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = gla.gated_ff_bwd(*static)
    for data in (inputs[0], small, inputs[1], small, inputs[0]):
        for t, d in zip(static, data):
            t.copy_(d)
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        want = gla.gated_ff_bwd(*data)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(outs, want))


@pytest.mark.parametrize("kind", ["silu", "gelu", "logsigmoid"])
@pytest.mark.parametrize("rows,K,N", [(5, 72, 24), (700, 72, 136)])
def test_linear_gradient_at_halfs_largest_values(rows, K, N, kind):
    """gy of 60,000 to 65,504 where the slopes are largest."""
    r = np.random.default_rng(rows)
    x, w = normal(r, np.float16, rows, K, s=2.0 ** -10), normal(r, np.float16, N, K, s=2.0 ** -11)
    gy = (np.linspace(60000, 65504, rows * N) * r.choice([-1, 1], rows * N)).astype(np.float16).reshape(rows, N)
    pre = np.linspace(0, 4, rows * N).astype(np.float16).reshape(rows, N) * (-1 if kind == "logsigmoid" else 1)
    pre = pre.astype(np.float16)
    got = gla.linear_bwd(*to_dev(x, w, gy), act=ACTS[kind], pre=to_dev(pre)[0])
    torch.cuda.synchronize()
    want = oracle.linear_backward(x, w, pre, gy, kind, 1.0)
    z = pre.astype(np.float64)
    gp = gy * oracle.act_slope(z, kind)
    assert kind == "logsigmoid" or np.abs(gp).max() > 65520  # would round to infinity
    slope_off = act_off(z) * np.abs(gy) * 1.13
    off = slope_off + half_step(np.float16, gp)
    A, W, X = np.abs(gp) + off, np.abs(w.astype(np.float64)), np.abs(x.astype(np.float64))
    check("gx", got[0], want[0], off @ W + sums(np.float16, N + 2, A @ W) + half_step(np.float16, want[0]))
    check("gweight", got[1], want[1], off.T @ X + sums(np.float16, rows + 2, A.T @ X) + half_step(np.float16, want[1]))
    check("gbias", got[2], want[2], slope_off.sum(0) + (rows + 4) * U * A.sum(0))


@pytest.mark.parametrize("kind", ["silu", "gelu", "logsigmoid"])
def test_sums_kept_beyond_halfs_range_have_slopes(kind):
    """pre of +-7e4 to 5e5 among ordinary ones: kept as infinities, behind an
    output that is finite; the slopes there are the limits."""
    r = np.random.default_rng(21)
    rows, K, N = 70, 72, 40
    x, w = normal(r, np.float16, rows, K), normal(r, np.float16, N, K, s=K ** -0.5)
    b = np.zeros(N, np.float32)
    b[:8] = np.linspace(7e4, 5e5, 8) * np.tile([1, -1], 4)
    gy = normal(r, np.float16, rows, N)
    dx, dw, db, dgy = to_dev(x, w, b, gy)
    y, pre = gla.linear(dx, dw, db, act=ACTS[kind], alpha=2.0 ** -6, return_pre=True)
    got = gla.linear_bwd(dx, dw, dgy, act=ACTS[kind], alpha=2.0 ** -6, pre=pre)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isinf(pre[:, :8]).all() and torch.isfinite(pre[:, 8:]).all()
    z = pre.double().cpu().numpy()
    z[:, :8] = oracle.linear(x, w, b)[0][:, :8]
    want = oracle.linear_backward(x, w, z, gy, kind, 2.0 ** -6)
    gp = gy * oracle.act_slope(z, kind)
    far = np.isinf(pre.double().cpu().numpy())
    slope_off = np.where(far, 0, act_off(np.where(far, 0, z)) * np.abs(gy) * 1.13)
    off = slope_off + half_step(np.float16, gp)
    A, W, X = np.abs(gp) + off, np.abs(w.astype(np.float64)), np.abs(x.astype(np.float64))
    c = 2.0 ** -6
    check("gx", got[0], want[0], c * (off @ W + sums(np.float16, N + 2, A @ W)) + half_step(np.float16, want[0]))
    check("gweight", got[1], want[1], c * (off.T @ X + sums(np.float16, rows + 2, A.T @ X)) + half_step(np.float16, want[1]))
    check("gbias", got[2], want[2], c * (slope_off.sum(0) + (rows + 4) * U * A.sum(0)) + 1e-30)
    nan = pre.clone()
    nan[3, 5] = float("nan")
    gx = gla.linear_bwd(dx, dw, dgy, act=ACTS[kind], pre=nan)[0]
    torch.cuda.synchronize()
    assert torch.isnan(gx[3]).all() and torch.isfinite(gx[:3]).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gates_kept_below_halfs_range_pass_nothing(kind):
    r = np.random.default_rng(22)
    rows, K, F = 70, 72, 40
    x, gh = normal(r, np.float16, rows, K), normal(r, np.float16, rows, F)
    wg, wu = (normal(r, np.float16, F, K, s=K ** -0.5) for _ in range(2))
    a, u = normal(r, np.float16, rows, F), normal(r, np.float16, rows, F)
    a[:, ::5] = -np.inf
    got = gla.gated_ff_bwd(*to_dev(x, wg, wu, a, u, gh), act=ACTS[kind])
    a[:, ::5] = -60000  # zero there, and as flat
    want = gla.gated_ff_bwd(*to_dev(x, wg, wu, a, u, gh), act=ACTS[kind])
    torch.cuda.synchronize()
    assert all(torch.isfinite(g).all() and torch.equal(g, t) for g, t in zip(got, want))
