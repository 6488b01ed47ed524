"""GPU: the norms after and before a block with its gate and residual scale, and
their gradient, against the float64 formulas.

Tolerance, u = 2^-24: a row's sums have at most 16 sequential additions per
thread, 10 joining ones and 16 over waves, n = 48 with room for the factors in
front; roots and products after them at most 8 more. So n(x) is off by n u of
itself, s by n u |scale gate p| + 2 u (|residual| + |s|) and half a step of the
type, y (of the kernel's own s) by n u |y| and half a step. In the gradient
mean(gy w m) is off by n u of its mean of magnitudes, so gS by
e = rs n u (|gy w| + |m| mean |gy w m|) + 2 u (|gS| + |gsum|). mean(gS f n) is
put together from three sums and off by n u of the sum of their magnitudes, E.
Sums over R rows: (R + n) u of the sum of magnitudes besides what the terms are
off by."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
U, EPS, NU = 2.0 ** -24, 1e-6, 48 * 2.0 ** -24
# (groups, rows per group, F): teams of every size, ends inside a team, one
# group, a group of every row's own, few and many groups
SHAPES = [(1, 1, 8), (3, 5, 40), (1, 70, 64), (2, 33, 72), (1, 9, 128), (5, 3, 136), (4, 50, 256), (1, 7, 264),
          (7, 1, 512), (3, 11, 520), (4, 130, 768), (1, 600, 1000), (2, 2, 1024), (3, 3, 1032), (1, 4, 4096),
          (2, 3, 4104), (1, 3, 8192), (2, 1, 8200), (1, 2, 16384), (1500, 1, 72), (1030, 3, 24), (1100, 2, 1032),
          (40, 9, 200)]
FORMS = [(1, 1, 1), (1, 0, 1), (0, 1, 0), (0, 0, 0), (1, 1, 0), (0, 1, 1)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def half_step(dtype, x):
    return 2.0 ** -11 * np.abs(x) + 2.0 ** -25 if dtype == np.float16 else U * np.abs(x)


def make(G, per, F, dtype, form, seed):
    r = np.random.default_rng(seed)
    n = lambda *s, m=1.0: (m * r.standard_normal(s)).astype(dtype)
    rows = G * per
    post, gated, scaled = form
    return dict(x=n(rows, F, m=2.0), res=n(rows, F, m=4.0), w=(1 + 0.1 * r.standard_normal(F)).astype(np.float32),
                post=(1 + 0.1 * r.standard_normal(F)).astype(np.float32) if post else None,
                gate=n(G, F) if gated else None,
                scale=(0.1 * r.standard_normal(F)).astype(np.float32) if scaled else None, gy=n(rows, F),
                gsum=n(rows, F))


def dev(d, *names):
    return [None if d[k] is None else to_dev(d[k])[0] for k in names]


def check(name, got, want, tol):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    worst = float(np.max(np.abs(got - want) / (tol + 1e-300)))
    say(f"  {name}: {worst:.3f} of the bound")
    assert worst <= 1, name


def run(d):
    x, res, w, post, gate, scale = dev(d, "x", "res", "w", "post", "gate", "scale")
    return gla.gated_add_rmsnorm(x, res, w, EPS, post_weight=post, gate=gate, scale=scale)


@pytest.mark.parametrize("G,per,F", SHAPES)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_forward(G, per, F, dtype):
    for form in FORMS:
        d = make(G, per, F, dtype, form, G + per + F)
        y, s = run(d)
        torch.cuda.synchronize()
        say(f"gated_add_rmsnorm {G}x{per}x{F} {np.dtype(dtype).name} post, gate, scale {form}")
        _, _, whole = oracle.gated_add_rmsnorm(d["x"], d["res"], d["w"], EPS, d["post"], d["gate"], d["scale"])
        add = np.abs(whole - d["res"].astype(np.float64))
        check("s", s, whole, NU * add + 4 * U * (np.abs(d["res"]) + np.abs(whole)) + half_step(dtype, whole))
        want, _ = oracle.add_rmsnorm(s.cpu().numpy(), None, d["w"], EPS)
        check("y", y, want, NU * np.abs(want) + half_step(dtype, want))


@pytest.mark.parametrize("G,per,F", SHAPES)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("carry", [True, False])
def test_backward(G, per, F, dtype, carry):
    for form in FORMS:
        d = make(G, per, F, dtype, form, G + per + F + 1)
        gsum = d["gsum"] if carry else None
        x, s, w, post, gate, scale, gy, gs = dev(d, "x", "res", "w", "post", "gate", "scale", "gy", "gsum")
        got = gla.gated_add_rmsnorm_bwd(x, s, w, EPS, gy, post_weight=post, gate=gate, scale=scale,
                                        gsum=gs if carry else None)
        torch.cuda.synchronize()
        say(f"gated_add_rmsnorm_bwd {G}x{per}x{F} {np.dtype(dtype).name} post, gate, scale {form} gsum {carry}")
        want = oracle.gated_add_rmsnorm_backward(d["x"], d["res"], d["w"], EPS, d["gy"], gsum, d["post"], d["gate"],
                                                 d["scale"])
        f64 = lambda a: np.asarray(a, np.float64)
        X, S, GY, W = f64(d["x"]), f64(d["res"]), f64(d["gy"]), f64(d["w"])
        mean = lambda a: np.mean(a, axis=-1, keepdims=True)
        rs = 1 / np.sqrt(mean(S * S) + EPS)
        rx = 1 / np.sqrt(mean(X * X) + EPS) if form[0] else np.ones_like(rs)
        m, n, gw = S * rs, X * rx, GY * W
        G0 = np.zeros_like(X) if gsum is None else f64(gsum)
        gate_rows = np.ones((1, 1)) if d["gate"] is None else np.repeat(f64(d["gate"]), per, 0)
        a = np.ones(F) if d["post"] is None else f64(d["post"])
        b = np.ones(F) if d["scale"] is None else f64(d["scale"])
        f = np.abs(a * b * gate_rows) * np.ones_like(X)
        dot = mean(np.abs(gw * m))
        e = rs * NU * (np.abs(gw) + np.abs(m) * dot) + 2 * U * (np.abs(want[1]) + np.abs(G0))
        E = NU * rx * mean(np.abs(G0 * f * X) + rs * np.abs(gw * f * X) + rs * rs * dot * np.abs(f * X * S))
        if not form[0]:
            E = 0 * E
        top = np.abs(want[1]) * f + np.abs(n) * (E / NU if form[0] else 0)
        check("gx", got[0], want[0], rx * (f * e + np.abs(n) * E + 16 * U * top) + half_step(dtype, want[0]))
        check("gresidual", got[1], want[1], e + half_step(dtype, want[1]))
        rows = G * per
        tw = (rows + 48) * U * np.abs(GY * m).sum(0) + half_step(np.float32, want[2])
        check("gweight", got[2], want[2], tw)
        q = np.abs(n) * e + (rows + 64) * U * np.abs(want[1] * n)
        if form[0]:
            check("gpost", got[3], want[3], (q * np.abs(b * gate_rows)).sum(0) + half_step(np.float32, want[3]))
        if form[1]:
            tg = (q * np.abs(a * b)).reshape(G, per, F).sum(1) + half_step(dtype, want[4])
            check("ggate", got[4], want[4], tg)
        if form[2]:
            check("gscale", got[5], want[5], (q * np.abs(a * gate_rows)).sum(0) + half_step(np.float32, want[5]))
        for g, t in zip(got, want):
            assert (g is None) == (t is None)


def test_without_gate_and_norms_it_is_add_rmsnorm():
    d = make(1, 50, 520, np.float16, (0, 0, 0), 3)
    x, res, w = dev(d, "x", "res", "w")
    a = gla.gated_add_rmsnorm(x, res, w, EPS)
    b = gla.add_rmsnorm(x, res, w, EPS)
    torch.cuda.synchronize()
    assert torch.equal(a[1], b[1])
    want, _ = oracle.add_rmsnorm(b[1].cpu().numpy(), None, d["w"], EPS)
    check("y", a[0], want, NU * np.abs(want) + half_step(np.float16, want))


def test_in_place():
    d = make(3, 20, 200, np.float16, (1, 1, 1), 5)
    x, res, w, post, gate, scale, gy, gs = dev(d, "x", "res", "w", "post", "gate", "scale", "gy", "gsum")
    kw = dict(post_weight=post, gate=gate, scale=scale)
    y, s = gla.gated_add_rmsnorm(x, res, w, EPS, **kw)
    x2, r2 = x.clone(), res.clone()
    y2, s2 = gla.gated_add_rmsnorm(x2, r2, w, EPS, out=x2, sum_out=r2, **kw)
    torch.cuda.synchronize()
    assert y2 is x2 and torch.equal(y, y2) and torch.equal(s, s2)
    want = gla.gated_add_rmsnorm_bwd(x, s, w, EPS, gy, gsum=gs, **kw)
    for which in range(4):
        t = [u.clone() for u in (x, s, gy, gs)]
        o = [t[which], t[(which + 1) % 4]]
        got = gla.gated_add_rmsnorm_bwd(t[0], t[1], w, EPS, t[2], gsum=t[3], gx=o[0], gresidual=o[1], **kw)
        torch.cuda.synchronize()
        assert got[0] is o[0] and all(torch.equal(p, q) for p, q in zip(got, want))


def test_gate_shapes_and_refusals():
    d = make(6, 4, 64, np.float16, (1, 1, 1), 6)
    x, res, w, post, gate, scale = dev(d, "x", "res", "w", "post", "gate", "scale")
    flat = gla.gated_add_rmsnorm(x, res, w, EPS, gate=gate)
    cube = lambda t: t.view(2, 3, 4, 64)
    y, s = gla.gated_add_rmsnorm(cube(x), cube(res), w, EPS, gate=gate.view(2, 3, 64))
    grads = gla.gated_add_rmsnorm_bwd(cube(x), s, w, EPS, y, gate=gate.view(2, 3, 64))
    torch.cuda.synchronize()
    assert torch.equal(cube(flat[0]), y) and grads[4].shape == (2, 3, 64) and grads[3] is None and grads[5] is None
    bad = [dict(gate=gate[:5].contiguous()), dict(gate=gate.float()), dict(gate=gate[:, :32]), dict(gate=gate[:0]),
           dict(scale=scale.half()), dict(post_weight=post[:8]), dict(scale=scale.cpu()), dict(out=x[:3]),
           dict(sum_out=torch.empty_like(x, device="cpu"))]
    for kw in bad:
        with pytest.raises(ValueError):
            gla.gated_add_rmsnorm(x, res, w, EPS, **kw)
    for call in (lambda: gla.gated_add_rmsnorm(x, res[:3], w, EPS), lambda: gla.gated_add_rmsnorm(x, res, w[:8], EPS),
                 lambda: gla.gated_add_rmsnorm_bwd(x, res, w, EPS, x[:3]),
                 lambda: gla.gated_add_rmsnorm_bwd(x, res, w, EPS, x, gsum=x.float())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gla.GLAError):
        gla.gated_add_rmsnorm(x, res, w, -1.0)
    with pytest.raises(gla.GLAError):  # a row's result beside its input
        gla.gated_add_rmsnorm(x[1:], res[1:], w, EPS, out=x[:-1])


def test_no_rows():
    w = torch.ones(64, device="cuda")
    none = torch.empty(0, 64, device="cuda").half()
    y, s = gla.gated_add_rmsnorm(none, none, w, EPS, post_weight=w, scale=w)
    g = gla.gated_add_rmsnorm_bwd(none, none, w, EPS, none, post_weight=w, scale=w)
    torch.cuda.synchronize()
    assert y.shape == s.shape == (0, 64) and g[0].shape == (0, 64)
    assert not g[2].any() and not g[3].any() and not g[5].any() and g[4] is None


def test_rows_keep_their_own_infinities():
    for F, G in ((64, 5), (768, 1), (5000, 5)):
        d = make(G, 15 // G, F, np.float16, (1, 1, 1), 8)
        clean = [t.cpu().numpy() for t in run(d)]
        for k, (row, col, v) in (("x", (3, 5, np.inf)), ("res", (7, 1, np.nan)), ("x", (11, 0, np.nan))):
            d[k][row, col] = v
        got = [t.cpu().numpy() for t in run(d)]
        ok = np.ones(15, bool)
        ok[[3, 7, 11]] = False
        for a, b in zip(got, clean):
            assert np.array_equal(a[ok], b[ok])
        assert np.isnan(got[0][7]).all() and np.isnan(got[0][11]).all() and np.isnan(got[1][7, 1])


def test_same_bits_every_time_on_streams_and_in_graphs():
    cases = [make(G, per, F, np.float16, (1, 1, 1), 9) for G, per, F in ((4, 100, 768), (1200, 2, 72))]
    ws = [torch.empty(32 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    moved = [dev(d, "x", "res", "w", "post", "gate", "scale", "gy", "gsum") for d in cases]

    def calls(k, stream=None):
        outs = []
        for x, res, w, post, gate, scale, gy, gs in moved:
            kw = dict(post_weight=post, gate=gate, scale=scale, stream=stream)
            outs += gla.gated_add_rmsnorm(x, res, w, EPS, **kw)
            outs += gla.gated_add_rmsnorm_bwd(x, res, w, EPS, gy, gsum=gs, workspace=ws[k], **kw)
        return outs

    first = calls(0)
    torch.cuda.synchronize()
    both = [calls(k, s) for k, s in enumerate((torch.cuda.Stream(), torch.cuda.Stream()))]
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
        again = calls(0)
        torch.cuda.synchronize()
        for outs in [o for _, o in graphs] + [again]:
            assert all(torch.equal(a, b) for a, b in zip(outs, first))


def test_workspace_need_is_enough():
    for G, per, F in ((1, 700, 768), (5, 40, 264), (1500, 1, 72), (1, 1, 8)):
        d = make(G, per, F, np.float32, (1, 1, 1), 10)
        x, res, w, post, gate, scale, gy = dev(d, "x", "res", "w", "post", "gate", "scale", "gy")
        need = gla.load().gla_gated_add_rmsnorm_bwd_workspace_bytes(G * per, G, F)
        room = torch.full((need + 8192,), 0xa5, dtype=torch.uint8, device="cuda")
        kw = dict(post_weight=post, gate=gate, scale=scale)
        want = gla.gated_add_rmsnorm_bwd(x, res, w, EPS, gy, **kw)
        got = gla.gated_add_rmsnorm_bwd(x, res, w, EPS, gy, workspace=room[4096:4096 + need], **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.all(room[:4096] == 0xa5) and torch.all(room[4096 + need:] == 0xa5)
