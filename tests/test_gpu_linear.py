"""GPU: linear products with their epilogue, the gated feed-forward product and
the gradients of both, against the float64 formulas.

Tolerances. Products of two halves are exact in float; a sum of K products in
any order is off by at most K u S with S the sum of magnitudes and u = 2^-23 for
each addition (one that truncates included), and the bias adds one more. For
float operands each product is rounded too: (K + 1) u S. An activation has slope
at most 1.13 and is itself off by (8 + |z| + z^2) 2^-22 of itself in float
(reciprocal, exp2, polynomial, and the rounding of the exponent). An output is
rounded once to its type: half a step. In the gradients the row gp behind the
activation is rounded to the type before the products: half a step of every
term, and for half 2^-25 below the smallest normal."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
ACTS = {"none": gla.ACT_NONE, "silu": gla.ACT_SILU, "gelu": gla.ACT_GELU, "logsigmoid": gla.ACT_LOGSIGMOID}
# one row, rows around the forms' borders (16, 32, 64), one and several tiles
# of both sizes, ends inside a tile and inside a step of the contraction
SHAPES = [(1, 8, 8), (1, 768, 136), (3, 72, 24), (16, 64, 40), (17, 200, 64), (33, 1032, 16), (64, 136, 264),
          (65, 64, 64), (65, 8, 8), (127, 72, 136), (130, 520, 72), (300, 40, 1000), (2100, 72, 2000),
          (4100, 136, 1032)]
SMALL = [(1, 8, 8), (3, 72, 24), (33, 136, 40), (65, 64, 64), (130, 520, 72), (700, 72, 136)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def half_step(dtype, x):
    return 2.0 ** -11 * np.abs(x) + 2.0 ** -25 if dtype == np.float16 else 2.0 ** -24 * np.abs(x)


def sums(dtype, K, S):
    """What a float sum of K products with magnitudes summing to S may be off by."""
    return (K + (2 if dtype == np.float32 else 1)) * U * S


def act_off(z):
    return (8 + np.abs(z) + z * z) * 2.0 ** -22


def normal(r, dtype, *shape, s=1.0):
    return (s * r.standard_normal(shape)).astype(dtype)


def check(name, got, want, tol):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    worst = float(np.max(np.abs(got - want) / tol))
    say(f"  {name}: {worst:.3f} of the bound")
    assert worst <= 1, name


def expect_linear(x, w, b, kind, alpha, res, dtype):
    """(y, its bound, pre, its bound)."""
    y, pre = oracle.linear(x, w, b, kind, alpha, res)
    S = np.abs(x.astype(np.float64)) @ np.abs(w.astype(np.float64)).T + (0 if b is None else np.abs(b))
    off = sums(dtype, x.shape[1], S)
    a = np.abs(oracle.act(pre, kind))
    ty = abs(alpha) * (1.13 * off + act_off(pre) * a) + 4 * U * (np.abs(y) + abs(alpha) * a) + half_step(dtype, y)
    return y, ty, pre, off + half_step(dtype, pre)


@pytest.mark.parametrize("rows,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_linear(rows, K, N, dtype):
    r = np.random.default_rng(rows + K + N)
    x, w, b = normal(r, dtype, rows, K), normal(r, dtype, N, K, s=K ** -0.5), normal(r, np.float32, N)
    res = normal(r, dtype, rows, N)
    dx, dw, db, dres = to_dev(x, w, b, res)
    y, ty, _, _ = expect_linear(x, w, None, "none", 1.0, None, dtype)
    got = gla.linear(dx, dw)
    full = {}
    for kind in ACTS:
        full[kind] = gla.linear(dx, dw, db, act=ACTS[kind], alpha=0.0625, residual=dres, return_pre=True)
    torch.cuda.synchronize()
    say(f"linear {rows}x{K}x{N} {np.dtype(dtype).name}")
    check("plain", got, y, ty)
    for kind, (gy, gpre) in full.items():
        y, ty, pre, tpre = expect_linear(x, w, b, kind, 0.0625, res, dtype)
        check(kind, gy, y, ty)
        check(kind + " pre", gpre, pre, tpre)


def test_linear_shapes_and_outputs_of_the_caller():
    r = np.random.default_rng(3)
    x, w, res = normal(r, np.float16, 2, 5, 64), normal(r, np.float16, 24, 64, s=0.125), normal(r, np.float16, 2, 5, 24)
    dx, dw, dres = to_dev(x, w, res)
    y = gla.linear(dx, dw, residual=dres)
    one = gla.linear(dx[0, 0].contiguous(), dw)
    keep = dres.clone()
    same = gla.linear(dx, dw, residual=keep, out=keep)  # the stream in place
    pre = torch.empty_like(dres)
    z, p = gla.linear(dx, dw, act=gla.ACT_SILU, return_pre=True, pre=pre)
    torch.cuda.synchronize()
    assert y.shape == (2, 5, 24) and one.shape == (24,) and same is keep and torch.equal(same, y)
    assert p is pre and torch.equal(pre, gla.linear(dx, dw))
    assert torch.equal(one, gla.linear(dx, dw)[0, 0])


@pytest.mark.parametrize("rows,K,F", SHAPES)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_gated_ff(rows, K, F, dtype):
    r = np.random.default_rng(rows + K + F + 1)
    x = normal(r, dtype, rows, K)
    wg, wu = (normal(r, dtype, F, K, s=K ** -0.5) for _ in range(2))
    dev = to_dev(x, wg, wu)
    say(f"gated_ff {rows}x{K}x{F} {np.dtype(dtype).name}")
    X = np.abs(x.astype(np.float64))
    oa, ou = (sums(dtype, K, X @ np.abs(w.astype(np.float64)).T) for w in (wg, wu))
    for kind in ("silu", "gelu"):
        h, a, u = oracle.gated_ff(x, wg, wu, kind)
        got, ga, gu = gla.gated_ff(*dev, act=ACTS[kind], return_parts=True)
        alone = gla.gated_ff(*dev, act=ACTS[kind])
        torch.cuda.synchronize()
        act = np.abs(oracle.act(a, kind))
        tol = (1.13 * oa + act_off(a) * act) * (np.abs(u) + ou) + act * ou + 2 * U * np.abs(h) + half_step(dtype, h)
        check(kind, got, h, tol)
        check("a", ga, a, oa + half_step(dtype, a))
        check("u", gu, u, ou + half_step(dtype, u))
        assert torch.equal(alone, got)


def gp_off(dtype, gp, z):
    """A row behind the activation: its slope in float, then rounded to the type."""
    return act_off(z) * (np.abs(gp) + 2.0 ** -24) + half_step(dtype, gp)


@pytest.mark.parametrize("rows,K,N", SMALL + [(2100, 1032, 136)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("kind", list(ACTS))
def test_linear_backward(rows, K, N, dtype, kind):
    r = np.random.default_rng(rows + K + N + 2)
    alpha = 0.5
    x, w, gy = normal(r, dtype, rows, K), normal(r, dtype, N, K, s=K ** -0.5), normal(r, dtype, rows, N)
    pre = normal(r, dtype, rows, N, s=2.0)
    dx, dw, dgy, dpre = to_dev(x, w, gy, pre)
    gx, gw, gb = gla.linear_bwd(dx, dw, dgy, act=ACTS[kind], alpha=alpha, pre=None if kind == "none" else dpre)
    torch.cuda.synchronize()
    say(f"linear_bwd {rows}x{K}x{N} {np.dtype(dtype).name} {kind}")
    want = oracle.linear_backward(x, w, pre, gy, kind, alpha)
    z = pre.astype(np.float64)
    gp = gy * oracle.act_slope(z, kind)
    slope_off = gy.astype(np.float64) * 0 if kind == "none" else act_off(z) * (np.abs(gy) * 1.13)
    off = slope_off + (0 if kind == "none" else half_step(dtype, gp))
    A, W, X = np.abs(gp) + off, np.abs(w.astype(np.float64)), np.abs(x.astype(np.float64))
    tx = alpha * (off @ W + sums(dtype, N, A @ W)) + U * np.abs(want[0]) + half_step(dtype, want[0])
    tw = alpha * (off.T @ X + sums(dtype, rows, A.T @ X)) + U * np.abs(want[1]) + half_step(dtype, want[1])
    tb = alpha * (slope_off.sum(0) + (rows + 4) * U * A.sum(0)) + half_step(np.float32, want[2])
    check("gx", gx, want[0], tx)
    check("gweight", gw, want[1], tw)
    assert gb.dtype == torch.float32
    check("gbias", gb, want[2], tb + 1e-30)


@pytest.mark.parametrize("rows,K,F", SMALL + [(2100, 264, 520)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_ff_backward(rows, K, F, dtype, kind):
    r = np.random.default_rng(rows + K + F + 3)
    x, gh = normal(r, dtype, rows, K), normal(r, dtype, rows, F)
    wg, wu = (normal(r, dtype, F, K, s=K ** -0.5) for _ in range(2))
    a, u = (normal(r, dtype, rows, F) for _ in range(2))
    got = gla.gated_ff_bwd(*to_dev(x, wg, wu, a, u, gh), act=ACTS[kind])
    torch.cuda.synchronize()
    say(f"gated_ff_bwd {rows}x{K}x{F} {np.dtype(dtype).name} {kind}")
    want = oracle.gated_ff_backward(x, wg, wu, a, u, gh, kind)
    z, v, g = (t.astype(np.float64) for t in (a, u, gh))
    ga, gu = g * v * oracle.act_slope(z, kind), g * oracle.act(z, kind)
    oa = act_off(z) * 1.13 * np.abs(g * v) + half_step(dtype, ga)
    ou = act_off(z) * np.abs(gu) + half_step(dtype, gu)
    A, B, X = np.abs(ga) + oa, np.abs(gu) + ou, np.abs(x.astype(np.float64))
    Wg, Wu = (np.abs(w.astype(np.float64)) for w in (wg, wu))
    tx = oa @ Wg + ou @ Wu + sums(dtype, 2 * F, A @ Wg + B @ Wu) + half_step(dtype, want[0])
    check("gx", got[0], want[0], tx)
    check("ggate_weight", got[1], want[1], oa.T @ X + sums(dtype, rows, A.T @ X) + half_step(dtype, want[1]))
    check("gup_weight", got[2], want[2], ou.T @ X + sums(dtype, rows, B.T @ X) + half_step(dtype, want[2]))


def test_gradients_that_are_not_wanted():
    r = np.random.default_rng(9)
    dx, dw, dgy, dpre, du = to_dev(*(normal(r, np.float16, *s) for s in ((70, 64), (40, 64), (70, 40), (70, 40), (70, 40))))
    full = gla.linear_bwd(dx, dw, dgy, act=gla.ACT_GELU, pre=dpre)
    for x, w, b in [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 0, 0)]:
        some = gla.linear_bwd(dx, dw, dgy, act=gla.ACT_GELU, pre=dpre, need_x=x, need_weight=w, need_bias=b)
        torch.cuda.synchronize()
        for got, want, wanted in zip(some, full, (x, w, b)):
            assert torch.equal(got, want) if wanted else got is None
    full = gla.gated_ff_bwd(dx, dw, dw, dpre, du, dgy)
    some = gla.gated_ff_bwd(dx, dw, dw, dpre, du, dgy, need_x=False)
    last = gla.gated_ff_bwd(dx, dw, dw, dpre, du, dgy, need_weights=False)
    torch.cuda.synchronize()
    assert some[0] is None and torch.equal(some[1], full[1]) and torch.equal(some[2], full[2])
    assert torch.equal(last[0], full[0]) and last[1] is None and last[2] is None


def test_no_rows_and_no_outputs():
    w, wg = torch.randn(24, 64, device="cuda").half(), torch.randn(0, 64, device="cuda").half()
    none = torch.empty(0, 64, device="cuda").half()
    assert gla.linear(none, w).shape == (0, 24)
    gx, gw, gb = gla.linear_bwd(none, w, torch.empty(0, 24, device="cuda").half())
    torch.cuda.synchronize()
    assert gx.shape == (0, 64) and not gw.any() and not gb.any() and gw.shape == (24, 64)
    x = torch.randn(3, 64, device="cuda").half()
    assert gla.linear(x, wg).shape == (3, 0) and gla.gated_ff(x, wg, wg).shape == (3, 0)
    gx, gw, gb = gla.linear_bwd(x, wg, torch.empty(3, 0, device="cuda").half())
    torch.cuda.synchronize()
    assert gx.shape == (3, 64) and not gx.any() and gw.shape == (0, 64) and gb.shape == (0,)


def test_refused_by_the_binding():
    x, w = torch.randn(4, 64, device="cuda").half(), torch.randn(24, 64, device="cuda").half()
    b = torch.zeros(24, device="cuda")
    bad = [lambda: gla.linear(x.t(), w), lambda: gla.linear(x, w.t()), lambda: gla.linear(x, w.float()),
           lambda: gla.linear(x, w.cpu()), lambda: gla.linear(x, w, b.half()), lambda: gla.linear(x, w, b[:8]),
           lambda: gla.linear(x, w, residual=x), lambda: gla.linear(x, w, out=x),
           lambda: gla.linear(x, w, pre=torch.empty(4, 24, device="cuda").half()),
           lambda: gla.linear(x, w[:, :32].contiguous()), lambda: gla.linear(x.cpu(), w),
           lambda: gla.linear_bwd(x, w, x), lambda: gla.linear_bwd(x, w, gla.linear(x, w), act=gla.ACT_SILU),
           lambda: gla.gated_ff(x, w, w[:8].contiguous()), lambda: gla.gated_ff(x, w, w, parts=[x, x]),
           lambda: gla.gated_ff_bwd(x, w, w, x, x, x)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        gla.linear(x.bfloat16(), w.bfloat16())
    for call in (lambda: gla.linear(x, w, act=4), lambda: gla.linear(x[:, :4].contiguous(), w[:, :4].contiguous())):
        with pytest.raises(gla.GLAError):
            call()


def test_activation_values_over_their_range():
    """z from -60 to 60 through a 1 x 1 product in float: tails and the middle."""
    z = np.concatenate([np.linspace(-60, 60, 4801), np.logspace(-30, -1, 400), -np.logspace(-30, -1, 399)])
    z = z[:len(z) // 8 * 8].astype(np.float32)
    x = np.zeros((1, 8), np.float32)
    x[0, 0] = 1
    w = np.zeros((len(z), 8), np.float32)
    w[:, 0] = z
    for kind in ("silu", "gelu", "logsigmoid"):
        y = gla.linear(*to_dev(x, w), act=ACTS[kind])
        torch.cuda.synchronize()
        want = oracle.act(z, kind)[None]
        check(kind, y, want, act_off(z.astype(np.float64)) * np.abs(want) + half_step(np.float32, want) + 2.0 ** -126 * 64)


def test_large_values_and_masked_garbage():
    """Infinities and NaN stay in the rows (and weights' columns) they are of;
    values beyond half's range come out infinite, half subnormals are kept."""
    for rows in (5, 70):
        r = np.random.default_rng(11)
        x, w = normal(r, np.float16, rows, 72), normal(r, np.float16, 40, 72)
        clean = gla.linear(*to_dev(x, w))
        x[2, 5], x[3, 7] = np.inf, np.nan
        w[9, 3] = np.nan
        got = gla.linear(*to_dev(x, w))
        torch.cuda.synchronize()
        ok = np.ones((rows, 40), bool)
        ok[2:4] = ok[:, 9] = False
        g, c = got.cpu().numpy(), clean.cpu().numpy()
        assert np.array_equal(g[ok], c[ok]) and np.isnan(g[3]).all() and np.isnan(g[:, 9]).all()
        assert not np.isfinite(g[2]).any()
        big = gla.linear(*to_dev(np.full((rows, 64), 60000, np.float16), np.ones((8, 64), np.float16)))
        tiny = gla.linear(*to_dev(np.full((rows, 64), 2.0 ** -24, np.float16), np.ones((8, 64), np.float16)))
        torch.cuda.synchronize()
        assert torch.isinf(big).all() and torch.all(tiny == 2.0 ** -18)


def test_same_bits_every_time_on_streams_and_in_graphs():
    r = np.random.default_rng(12)
    x, w, gy = normal(r, np.float16, 700, 136), normal(r, np.float16, 264, 136, s=0.1), normal(r, np.float16, 700, 264)
    pre, u = normal(r, np.float16, 700, 264), normal(r, np.float16, 700, 264)
    dx, dw, dgy, dpre, du = to_dev(x, w, gy, pre, u)
    ws = [torch.empty(64 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def calls(k, stream=None):
        return (*gla.linear(dx, dw, act=gla.ACT_SILU, return_pre=True, stream=stream),
                *gla.linear_bwd(dx, dw, dgy, act=gla.ACT_SILU, pre=dpre, workspace=ws[k], stream=stream),
                *gla.gated_ff(dx, dw, dw, return_parts=True, stream=stream),
                *gla.gated_ff_bwd(dx, dw, dw, dpre, du, dgy, workspace=ws[k], stream=stream),
                gla.linear(dx[:40], dw, stream=stream), gla.gated_ff(dx[:7], dw, dw, stream=stream))

    first = calls(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [calls(k, s) for k, s in enumerate(streams)]  # at once, a workspace each
    torch.cuda.synchronize()
    for outs in both:
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = calls(k)
        graphs.append((g, outs))
    for _ in range(3):
        for g, outs in graphs:
            for t in outs:
                t.fill_(float("nan"))
            g.replay()
        again = calls(0)  # eager work between the replays
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, first))
        assert all(torch.equal(a, b) for a, b in zip(again, first))


def test_memory_behind_the_outputs_is_left_alone():
    r = np.random.default_rng(13)
    for rows in (5, 130):
        x, w, gy = (to_dev(normal(r, np.float16, *s))[0] for s in ((rows, 72), (40, 72), (rows, 40)))
        room = torch.full((4, rows * 72 + 4096), 7.0, device="cuda").half()
        y, gx = room[0, :rows * 40].view(rows, 40), room[1, :rows * 72].view(rows, 72)
        gw, h = room[2, :40 * 72].view(40, 72), room[3, :rows * 40].view(rows, 40)
        gla.linear(x, w, out=y)
        gla.linear_bwd(x, w, gy, gx=gx, gweight=gw)
        gla.gated_ff(x, w, w, out=h)
        torch.cuda.synchronize()
        for k, n in enumerate((rows * 40, rows * 72, 40 * 72, rows * 40)):
            assert torch.all(room[k, n:] == 7), k


def test_workspace_need_is_enough():
    """A workspace of exactly the stated size, of any contents, between guards."""
    r = np.random.default_rng(14)
    for rows, K, N in ((65, 64, 64), (3000, 72, 136)):
        dx, dw, dgy, dpre = to_dev(*(normal(r, np.float16, *s) for s in ((rows, K), (N, K), (rows, N), (rows, N))))
        lib = gla.load()
        for need, call in ((lib.gla_linear_bwd_workspace_bytes(rows, K, N, 1, 0),
                            lambda ws: gla.linear_bwd(dx, dw, dgy, act=gla.ACT_SILU, pre=dpre, workspace=ws)),
                           (lib.gla_gated_ff_bwd_workspace_bytes(rows, K, N, 0),
                            lambda ws: gla.gated_ff_bwd(dx, dw, dw, dpre, dgy, dgy, workspace=ws))):
            want = call(None)
            room = torch.full((need + 8192,), 0xa5, dtype=torch.uint8, device="cuda")
            got = call(room[4096:4096 + need])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert torch.all(room[:4096] == 0xa5) and torch.all(room[4096 + need:] == 0xa5)
