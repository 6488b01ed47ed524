"""GPU: the products and norms between a block's mixers at the edges of what they
take: empty batches, sums and gradients at and beyond half's range on their way, rows
near the ends of float's range, wide rows with many groups, the borders of the
form for few rows, slopes far out and where they cross zero.

Tolerances are those of test_gpu_linear.py."""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_gated_norm as norms
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla
from test_gpu_linear import ACTS, U, act_off, check, expect_linear, half_step, normal, sums

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


# one tile, both products in one launch and in two, the weights' rows split
@pytest.mark.parametrize("rows,K,F", [(1, 8, 8), (3, 72, 24), (65, 64, 64), (700, 72, 136), (2100, 264, 520),
                                      (5000, 520, 1032)])
@pytest.mark.parametrize("kind", ["silu", "gelu", "none"])
def test_gated_gradient_up_to_halfs_range_on_the_way(rows, K, F, kind):
    """ga and gu of up to 65,504, and none beyond."""
    r = np.random.default_rng(rows + K + F + 4)
    x = normal(r, np.float16, rows, K, s=2.0 ** -10)
    wg, wu = (normal(r, np.float16, F, K, s=2.0 ** -11) for _ in range(2))
    a, u = normal(r, np.float16, rows, F, s=3.0), normal(r, np.float16, rows, F, s=300.0)
    gh = r.uniform(-1, 1, (rows, F))
    z, v = a.astype(np.float64), u.astype(np.float64)
    slope, act = oracle.act_slope(z, kind), oracle.act(z, kind)
    gh = (gh * 65400 / np.maximum(np.abs(v * slope), np.maximum(np.abs(act), 1.0))).astype(np.float16)
    gh[0, 0], u[0, 0], a[0, 0] = 65, 1000, 20  # 65,000, as the slope is 1
    z, v, g = (t.astype(np.float64) for t in (a, u, gh))
    ga, gu = g * v * oracle.act_slope(z, kind), g * oracle.act(z, kind)
    assert 64900 < max(np.abs(ga).max(), np.abs(gu).max()) <= 65504
    got = gla.gated_ff_bwd(*to_dev(x, wg, wu, a, u, gh), act=ACTS[kind])
    torch.cuda.synchronize()
    say(f"gated_ff_bwd {rows}x{K}x{F} {kind}, large")
    want = oracle.gated_ff_backward(x, wg, wu, a, u, gh, kind)
    assert all(np.abs(w).max() < 60000 for w in want)
    step = lambda t: half_step(np.float16, t)
    off = 0 * z if kind == "none" else act_off(z)
    oa, ou = off * 1.13 * np.abs(g * v) + 4 * U * np.abs(ga) + step(ga), off * np.abs(gu) + 4 * U * np.abs(gu) + step(gu)
    A, B, X = np.abs(ga) + oa, np.abs(gu) + ou, np.abs(x.astype(np.float64))
    Wg, Wu = (np.abs(w.astype(np.float64)) for w in (wg, wu))
    check("gx", got[0], want[0], oa @ Wg + ou @ Wu + sums(np.float16, 2 * F, A @ Wg + B @ Wu) + step(want[0]))
    for name, k, o, t in (("ggate_weight", 1, oa, A), ("gup_weight", 2, ou, B)):
        check(name, got[k], want[k], o.T @ X + sums(np.float16, rows, t.T @ X) + step(want[k]))


@pytest.mark.parametrize("rows,K,F", [(70, 72, 40), (5000, 520, 1032)])
def test_a_gated_gradient_beyond_halfs_range_stays_in_its_rows(rows, K, F):
    """gh u act'(a) of 1e6 is infinite in half: in its row of gx and of the gate
    weight's gradient, and nowhere else."""
    r = np.random.default_rng(17)
    x, gh = normal(r, np.float16, rows, K), normal(r, np.float16, rows, F)
    wg, wu = (normal(r, np.float16, F, K, s=K ** -0.5) for _ in range(2))
    a, u = normal(r, np.float16, rows, F), normal(r, np.float16, rows, F)
    a[3, 5], u[3, 5], gh[3, 5] = 20, 1000, 0
    want = gla.gated_ff_bwd(*to_dev(x, wg, wu, a, u, gh))
    gh[3, 5] = 1000
    got = gla.gated_ff_bwd(*to_dev(x, wg, wu, a, u, gh))
    torch.cuda.synchronize()
    row, col = np.arange(rows) != 3, np.arange(F) != 5
    assert not torch.isfinite(got[0][3]).any() and not torch.isfinite(got[1][5]).any()
    assert torch.equal(got[0][row], want[0][row]) and all(torch.equal(got[k][col], want[k][col]) for k in (1, 2))
    assert torch.isfinite(got[2]).all() and not torch.equal(got[2][5], want[2][5])


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


def norm_gradient_bounds(d, want, eps, gsum=True):
    """Bounds of test_gpu_gated_norm.py for (gx, gresidual, gweight, gpost, ggate, gscale) of one group a row or
    one for all, with post, gate and scale. The sums that meet in mean(gS f n) are of the same values, so they are
    off by as much of their magnitudes."""
    NU, u = norms.NU, norms.U
    f64 = lambda a: np.asarray(a, np.float64)
    X, S, GY, W = f64(d["x"]), f64(d["res"]), f64(d["gy"]), f64(d["w"])
    G0 = f64(d["gsum"]) if gsum else np.zeros_like(X)
    mean = lambda a: np.mean(a, axis=-1, keepdims=True)
    rs, rx = 1 / np.sqrt(mean(S * S) + eps), 1 / np.sqrt(mean(X * X) + eps)
    m, n, gw = S * rs, X * rx, GY * W
    rows, F = X.shape
    per = rows // len(d["gate"])
    gate = np.repeat(f64(d["gate"]), per, 0)
    a, b = f64(d["post"]), f64(d["scale"])
    f = np.abs(a * b * gate)
    dot = mean(np.abs(gw * m))
    e = rs * NU * (np.abs(gw) + np.abs(m) * dot) + 2 * u * (np.abs(want[1]) + np.abs(G0))
    E = NU * mean(np.abs(G0 * f * n) + rs * np.abs(gw * f * n) + rs * dot * np.abs(f * n * m))
    half = (lambda x: half_step(np.float16, x)) if d["x"].dtype == np.float16 else (lambda x: 2.0 ** -24 * np.abs(x))
    low = 0 if d["x"].dtype == np.float16 else 2.0 ** -149
    top = np.abs(want[1]) * f + np.abs(n) * E / NU
    q = np.abs(n) * e + (rows + 64) * u * np.abs(want[1] * n)
    fine = lambda x: 2.0 ** -24 * np.abs(x) + low
    return (rx * (f * e + np.abs(n) * E + 16 * u * top) + half(want[0]) + low, e + half(want[1]) + low,
            (rows + 48) * u * np.abs(GY * m).sum(0) + fine(want[2]),
            (q * np.abs(b * gate)).sum(0) + fine(want[3]),
            (q * np.abs(a * b)).reshape(len(d["gate"]), per, F).sum(1) + half(want[4]) + low,
            (q * np.abs(a * gate)).sum(0) + fine(want[5]))


def hold_norm_gradient(d, eps):
    x, s, w, post, gate, scale, gy, gs = norms.dev(d, "x", "res", "w", "post", "gate", "scale", "gy", "gsum")
    got = gla.gated_add_rmsnorm_bwd(x, s, w, eps, gy, post_weight=post, gate=gate, scale=scale, gsum=gs)
    torch.cuda.synchronize()
    want = oracle.gated_add_rmsnorm_backward(d["x"], d["res"], d["w"], eps, d["gy"], d["gsum"], d["post"], d["gate"],
                                             d["scale"])
    for name, g, t, tol in zip(("gx", "gresidual", "gweight", "gpost", "ggate", "gscale"), got, want,
                               norm_gradient_bounds(d, want, eps)):
        check(name, g, t, tol)


# x, s, scale, gy and gsum times these: a product of two of them is beyond float's range, or far below its normal
# values, where mean(x^2) and mean(s^2) are normal floats and every gradient is in range
@pytest.mark.parametrize("x,s,scale,gy,gsum", [(1e16, 1e16, 1e8, 1, 1e-16), (1e-17, 1e-17, 1, 1e-22, 1e-5),
                                               (1, 1e15, 1, 1e25, 1e10), (1e15, 1, 1, 1, 1e25), (1e-15, 1, 1, 1e-25, 1e-25)])
@pytest.mark.parametrize("G,per,F", [(3, 5, 40), (4, 50, 256), (2, 30, 768), (2, 3, 2056), (2, 3, 4104), (2, 3, 8200),
                                     (600, 1, 72)])
def test_norms_gradient_of_floats_near_their_ends(x, s, scale, gy, gsum, G, per, F):
    d = norms.make(G, per, F, np.float32, (1, 1, 1), G + per + F + 5)
    for name, c in (("x", x), ("res", s), ("scale", scale), ("gy", gy), ("gsum", gsum)):
        d[name] = d[name] * np.float32(c)
    hold_norm_gradient(d, 0.0 if min(x, s) < 1 else EPS)


# rows of every width that has a kernel of its own, with a gate of every row's own, of two rows', and chunks of a group
@pytest.mark.parametrize("G,per,F", [(520, 1, 4104), (512, 2, 4104), (515, 1, 8192), (520, 1, 8200), (512, 2, 8200),
                                     (514, 1, 16384), (3, 200, 8200), (1, 600, 16384), (20, 3, 8200),
                                     (300, 1, 8200)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_norms_of_wide_rows_with_many_groups(G, per, F, dtype):
    d = norms.make(G, per, F, dtype, (1, 1, 1), G + per + F + 6)
    hold_norm_gradient(d, EPS)
    y, s = norms.run(d)
    torch.cuda.synchronize()
    _, _, whole = oracle.gated_add_rmsnorm(d["x"], d["res"], d["w"], EPS, d["post"], d["gate"], d["scale"])
    add = np.abs(whole - d["res"].astype(np.float64))
    check("s", s, whole, norms.NU * add + 4 * norms.U * (np.abs(d["res"]) + np.abs(whole)) + norms.half_step(dtype, whole))
    want, _ = oracle.add_rmsnorm(s.cpu().numpy(), None, d["w"], EPS)
    check("y", y, want, norms.NU * np.abs(want) + norms.half_step(dtype, want))
    alone = gla.gated_add_rmsnorm_bwd(*norms.dev(d, "x", "res", "w"), EPS, *norms.dev(d, "gy"))
    torch.cuda.synchronize()
    plain = dict(d, post=np.ones(F, np.float32), gate=np.ones((1, F), dtype), scale=np.ones(F, np.float32))
    want = oracle.gated_add_rmsnorm_backward(d["x"], d["res"], d["w"], EPS, d["gy"])
    tol = norm_gradient_bounds(plain, want[:3] + (want[2],) * 3, EPS, gsum=False)
    for name, k in (("gresidual alone", 1), ("gweight alone", 2)):
        check(name, alone[k], want[k], tol[k])
    check("gx alone", alone[0], want[0], tol[1])  # the same values


@pytest.mark.parametrize("rows", [1, 4, 5, 16, 17])
@pytest.mark.parametrize("N", [2056, 4096, 4104, 8192, 8200, 16392])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_few_rows_with_many_outputs(rows, N, dtype):
    K = 136
    r = np.random.default_rng(rows + N + 7)
    x, w, v = normal(r, dtype, rows, K), normal(r, dtype, N, K, s=K ** -0.5), normal(r, dtype, N, K, s=K ** -0.5)
    b, res = normal(r, np.float32, N), normal(r, dtype, rows, N)
    dx, dw, dv, db, dres = to_dev(x, w, v, b, res)
    y, ty, pre, tpre = expect_linear(x, w, b, "silu", 0.5, res, dtype)
    got, gpre = gla.linear(dx, dw, db, act=gla.ACT_SILU, alpha=0.5, residual=dres, return_pre=True)
    h, a, u = gla.gated_ff(dx, dw, dv, return_parts=True)
    torch.cuda.synchronize()
    check("linear", got, y, ty)
    check("pre", gpre, pre, tpre)
    X = np.abs(x.astype(np.float64))
    oa, ou = (sums(dtype, K, X @ np.abs(m.astype(np.float64)).T) for m in (w, v))
    rh, ra, ru = oracle.gated_ff(x, w, v, "silu")
    act = np.abs(oracle.act(ra, "silu"))
    check("a", a, ra, oa + half_step(dtype, ra))
    check("u", u, ru, ou + half_step(dtype, ru))
    check("h", h, rh, (1.13 * oa + act_off(ra) * act) * (np.abs(ru) + ou) + act * ou + 2 * U * np.abs(rh) +
          half_step(dtype, rh))


@pytest.mark.parametrize("kind", ["silu", "gelu", "logsigmoid"])
def test_slopes_over_their_range(kind):
    """The bias's gradient of one row with gy 1 is the slope in float: from -100 to
    100, close to where silu' and gelu' cross zero, next to 0 and at float's ends,
    to the bound of the two terms that it is the sum of. A sigmoid or a bell below
    2^-126 counts as zero, and at |z| <= 128 makes up to 2^-119."""
    z = np.concatenate([np.linspace(-100, 100, 8001), np.linspace(-1.2785, -1.2784, 500), np.linspace(-0.752, -0.7517, 500),
                        np.logspace(-30, -1, 400), -np.logspace(-30, -1, 400), [1e4, -1e4, 3e38, -3e38]])
    z = z[len(z) % 8:].astype(np.float32)
    N = len(z)
    zeros = torch.zeros(N, 8, device="cuda")
    gb = gla.linear_bwd(zeros[:1], zeros, torch.ones(1, N, device="cuda"), act=ACTS[kind], pre=to_dev(z[None])[0],
                        need_x=False, need_weight=False)[2]
    torch.cuda.synchronize()
    x = z.astype(np.float64)
    want = oracle.act_slope(x, kind)
    s = np.exp(-np.logaddexp(0, -x))
    phi = np.exp(-np.minimum(np.abs(x), 1e3) ** 2 / 2) / np.sqrt(2 * np.pi)
    terms = {"silu": s + np.abs(x) * s * np.exp(-np.logaddexp(0, x)), "gelu": np.abs(want - x * phi) + np.abs(x) * phi,
             "logsigmoid": want}[kind]
    check(kind, gb, want, act_off(np.minimum(np.abs(x), 128)) * terms + 2.0 ** -24 * np.abs(want) + 2.0 ** -119)


@pytest.mark.parametrize("G,per,F", [(3, 4, 8200), (515, 1, 8200), (512, 2, 8200), (513, 1, 4104)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_wide_rows_in_place_and_in_their_workspace(G, per, F, dtype):
    """gx and gresidual in each of the rows that they are made from, in a workspace
    of exactly the stated size between guards."""
    d = norms.make(G, per, F, dtype, (1, 1, 1), G + per + F + 8)
    x, res, w, post, gate, scale, gy, gs = norms.dev(d, "x", "res", "w", "post", "gate", "scale", "gy", "gsum")
    kw = dict(post_weight=post, gate=gate, scale=scale)
    y, s = gla.gated_add_rmsnorm(x, res, w, EPS, **kw)
    x2, r2 = x.clone(), res.clone()
    gla.gated_add_rmsnorm(x2, r2, w, EPS, out=x2, sum_out=r2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, x2) and torch.equal(s, r2)
    want = gla.gated_add_rmsnorm_bwd(x, s, w, EPS, gy, gsum=gs, **kw)
    need = gla.load().gla_gated_add_rmsnorm_bwd_workspace_bytes(G * per, G, F)
    assert need <= 2 * 4 * F * 1024
    room = torch.full((need + 8192,), 0xa5, dtype=torch.uint8, device="cuda")
    for which in range(4):
        t = [u.clone() for u in (x, s, gy, gs)]
        got = gla.gated_add_rmsnorm_bwd(t[0], t[1], w, EPS, t[2], gsum=t[3], gx=t[which], gresidual=t[(which + 1) % 4],
                                        workspace=room[4096:4096 + need], **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert torch.all(room[:4096] == 0xa5) and torch.all(room[4096 + need:] == 0xa5)
