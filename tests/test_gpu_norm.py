"""GPU: residual addition with RMS norm (in the input type and in 8 bits), its
gradient, and the output gate's gradient, against the float64 formulas.

Tolerance, u = 2^-24: a row's sum of squares has at most F/64 sequential float
additions per lane and 6 + 2 joining ones (n = F/64 + 8), its root and the
factors after it at most 8 more roundings: y off by (n + 8) u of |y| plus half a
step of the type. A gradient subtracts n mean(gn n), whose sum is off by the
same share of mean |gn n|: rstd (2n + 16) u (|gn| + |n| mean |gn n|). Weight
gradients add rows: at most R sequential additions, (R + n + 16) u of the sum of
magnitudes. In 8 bits a value is off by half a step of e4m3, at most 2^-4 of
itself or 2^-10 below the smallest normal, of the scale's 448ths; near a tie
the float error may move it one step, so the bar is on y8 * scale against y,
with (n + 8) u added; the largest value of a row is 448 exactly."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
WIDTHS = [(1, 8), (3, 40), (5, 512), (7, 520), (130, 768), (4, 1000), (2, 1024), (9, 2048), (3, 2056),
          (2, 4096), (2, 4104), (1, 8192), (3, 8200), (2, 16384)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def half_step(dtype, x):
    return 2.0 ** -11 * np.abs(x) + 2.0 ** -25 if dtype == np.float16 else U * np.abs(x)


def make(rows, F, dtype, seed):
    r = np.random.default_rng(seed)
    return (r.standard_normal((rows, F)).astype(dtype), (4 * r.standard_normal((rows, F))).astype(dtype),
            (1 + 0.1 * r.standard_normal(F)).astype(np.float32), r.standard_normal((rows, F)).astype(dtype),
            r.standard_normal((rows, F)).astype(dtype))


@pytest.mark.parametrize("rows,F", WIDTHS)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("with_res", [True, False])
def test_add_rmsnorm(rows, F, dtype, with_res):
    x, r, w, _, _ = make(rows, F, dtype, F + rows)
    res = r if with_res else None
    want, s = oracle.add_rmsnorm(x, res, w, EPS)
    dx, dr, dw = to_dev(x, r, w)
    y, ds = gla.add_rmsnorm(dx, dr if with_res else None, dw, EPS)
    torch.cuda.synchronize()
    tol = (F / 64 + 16) * U * np.abs(want) + half_step(dtype, want)
    worst = float(np.max(np.abs(y.double().cpu().numpy() - want) / tol))
    say(f"addnorm {rows}x{F} {np.dtype(dtype).name} residual={with_res}: {worst:.3f} of the bound")
    assert worst <= 1 and np.array_equal(ds.double().cpu().numpy(), s)


@pytest.mark.parametrize("rows,F", WIDTHS)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_add_rmsnorm_q8(rows, F, dtype):
    x, r, w, _, _ = make(rows, F, dtype, F + rows + 1)
    want, s = oracle.add_rmsnorm(x, r, w, EPS)
    y8, sc, ds = gla.add_rmsnorm_q8(*to_dev(x, r, w), EPS)
    torch.cuda.synchronize()
    assert y8.dtype == torch.float8_e4m3fn and sc.shape == (rows,)
    code, scale = y8.float().cpu().numpy().astype(np.float64), sc.double().cpu().numpy()
    n = F / 64 + 16
    top = np.max(np.abs(want), 1)
    assert np.max(np.abs(scale - top / 448) / (top / 448)) <= (n + 2) * U
    assert np.all(np.max(np.abs(code), 1) == 448)
    assert np.all(np.isin(np.abs(code), oracle.e4m3_values()))
    q = want / scale[:, None]
    tol = np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10) + (n + 4) * U * np.abs(q)
    worst = float(np.max(np.abs(code - q) / tol))
    # away from ties the nearest value is the only right one
    v = oracle.e4m3_values()
    mid = (v[1:] + v[:-1]) / 2
    near = np.abs(np.abs(q)[..., None] - mid).min(-1) <= (n + 4) * U * np.abs(q) if q.size <= 200000 else np.zeros_like(q, bool)
    nearest = v[np.searchsorted(mid, np.abs(q))] * np.sign(q)
    say(f"addnorm8 {rows}x{F} {np.dtype(dtype).name}: {worst:.3f} of the bound, {int(near.sum())} at ties")
    assert worst <= 1 and np.array_equal(ds.double().cpu().numpy(), s)
    if q.size <= 200000:
        assert np.array_equal(code[~near], nearest[~near])


def test_q8_rows_of_zeros_and_tiny_rows():
    x = np.zeros((3, 64), np.float32)
    x[1] = 1e-30
    x[2, 5] = 3.0
    y8, sc, _ = gla.add_rmsnorm_q8(*to_dev(x), None, torch.ones(64, device="cuda"), EPS)
    torch.cuda.synchronize()
    code = y8.float().cpu().numpy()
    assert np.all(code[0] == 0) and sc[0].item() == 1.0
    assert np.isfinite(code).all() and code[2, 5] == 448 and np.all(code[1] == 448)
    assert abs(sc[1].item() / (1e-27 / 448) - 1) < 1e-5  # 1e-30 / sqrt(1e-6): eps rules


def test_no_sum_output_and_in_place():
    lib = gla.load()
    x, r, w, _, _ = make(6, 200, np.float16, 5)
    dx, dr, dw = to_dev(x, r, w)
    want_y, want_s = gla.add_rmsnorm(dx, dr, dw, EPS)
    y = torch.empty_like(dx)
    torch.cuda.synchronize()
    st = torch.cuda.current_stream().cuda_stream
    assert lib.gla_add_rmsnorm(dx.data_ptr(), dr.data_ptr(), dw.data_ptr(), EPS, None, y.data_ptr(), 6, 200, 0, st) == gla.OK
    torch.cuda.synchronize()
    assert torch.equal(y, want_y)
    a, b = dx.clone(), dr.clone()
    ya, sa = gla.add_rmsnorm(a, b, dw, EPS, out=a, sum_out=b)  # the residual stream in place
    torch.cuda.synchronize()
    assert torch.equal(ya, want_y) and torch.equal(sa, want_s)


@pytest.mark.parametrize("rows,F", WIDTHS + [(4500, 64), (5000, 768)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("carry", [True, False])
def test_norm_gradient(rows, F, dtype, carry):
    _, s, w, gy, gs = make(rows, F, dtype, F + rows + 2)
    want, ww = oracle.add_rmsnorm_backward(s, w, EPS, gy, gs if carry else None)
    ds, dw, dgy, dgs = to_dev(s, w, gy, gs)
    gx, gw = gla.add_rmsnorm_bwd(ds, dw, EPS, dgy, gsum=dgs if carry else None)
    torch.cuda.synchronize()
    s6, g6 = s.astype(np.float64), gy.astype(np.float64)
    rstd = 1 / np.sqrt(np.mean(s6 * s6, 1, keepdims=True) + EPS)
    nn, gn = s6 * rstd, g6 * w
    n = F / 64 + 8
    mag = rstd * (np.abs(gn) + np.abs(nn) * np.mean(np.abs(gn * nn), 1, keepdims=True))
    tol = (2 * n + 16) * U * mag + 2 * U * np.abs(gs if carry else 0) + half_step(dtype, want)
    worst = float(np.max(np.abs(gx.double().cpu().numpy() - want) / tol))
    tw = (rows + n + 16) * U * np.sum(np.abs(g6 * nn), 0) + 1e-37
    ww_worst = float(np.max(np.abs(gw.double().cpu().numpy() - ww) / tw))
    say(f"normbwd {rows}x{F} {np.dtype(dtype).name} carry={carry}: gx {worst:.3f}, gweight {ww_worst:.3f} of the bound")
    assert worst <= 1 and ww_worst <= 1


def test_norm_gradient_in_place_and_repeatable():
    _, s, w, gy, gs = make(777, 768, np.float16, 8)
    ds, dw, dgy, dgs = to_dev(s, w, gy, gs)
    gx, gw = gla.add_rmsnorm_bwd(ds, dw, EPS, dgy, gsum=dgs)
    torch.cuda.synchronize()
    for i in range(3):
        a = [ds.clone(), dgy.clone(), dgs.clone()]
        x, y = gla.add_rmsnorm_bwd(a[0], dw, EPS, a[1], gsum=a[2], out=a[i])
        torch.cuda.synchronize()
        assert torch.equal(x, gx) and torch.equal(y, gw)


@pytest.mark.parametrize("dv", [32, 64])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 7, 3), (2, 33, 5), (3, 700, 4), (1, 6400, 6)])
def test_gate_gradient(shape, dv, dtype):
    r = np.random.default_rng(sum(shape) + dv)
    o = (2 * r.standard_normal(shape + (dv,))).astype(dtype)
    z, gy = ((3 * r.standard_normal(shape + (dv,))).astype(dtype) for _ in range(2))
    w = (1 + 0.1 * r.standard_normal(dv)).astype(np.float32)
    want = oracle.rmsnorm_gate_backward(o, z, w, EPS, gy)
    got = gla.gate_bwd(*to_dev(o, z, w), EPS, *to_dev(gy))
    torch.cuda.synchronize()
    o6, z6, g6 = (a.astype(np.float64) for a in (o, z, gy))
    rstd = 1 / np.sqrt(np.mean(o6 * o6, -1, keepdims=True) + EPS)
    nn, act = o6 * rstd, oracle.silu(z6)
    gn = g6 * w * act
    m = rstd * (np.abs(gn) + np.abs(nn) * np.mean(np.abs(gn * nn), -1, keepdims=True))
    sig = 1 / (1 + np.exp(-z6))
    # exp's argument z log2 e is rounded once: its value is off by (2 + |z|) u
    e = 32 + 2 * np.abs(z6)
    rows = int(np.prod(shape))
    tols = (np.max(e, -1, keepdims=True) * U * m + half_step(dtype, want[0]),
            2 * e * U * np.abs(g6 * nn * w) * (sig + np.abs(z6) * sig * (1 - sig)) + 4 * U * np.abs(z6 * g6 * nn * w * sig) + half_step(dtype, want[1]),
            (rows + np.max(e)) * U * np.sum(np.abs(g6 * nn * act).reshape(-1, dv), 0) + 1e-37)
    for name, a, b, t in zip(("go", "ggate", "gnorm_weight"), got, want, tols):
        worst = float(np.max(np.abs(a.double().cpu().numpy() - b) / t))
        say(f"gatebwd {shape} dv={dv} {np.dtype(dtype).name} {name}: {worst:.3f} of the bound")
        assert worst <= 1, name


def test_gate_gradient_far_gates():
    """silu's flat ends: gates of +-60000 give finite gradients, 0 or 1."""
    z = torch.tensor([[60000.0, -60000.0] * 16], dtype=torch.float16, device="cuda")
    o, gy, w = torch.ones_like(z), torch.ones_like(z), torch.ones(32, device="cuda")
    go, gz, gw = gla.gate_bwd(o, z, w, EPS, gy)
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(t).all()) for t in (go, gz, gw))
    assert bool((gz[0, 0::2] == 1).all()) and bool((gz[0, 1::2] == 0).all())


def test_graph_replays_with_eager_work_between():
    x, r, w, gy, gs = make(600, 768, np.float16, 9)
    dx, dr, dw, dgy, dgs = to_dev(x, r, w, gy, gs)
    o, z = dx.view(600, 12, 64), dr.view(600, 12, 64)
    gyo = dgy.view(600, 12, 64)
    nw = dw[:64].contiguous()

    def call():
        y, s = gla.add_rmsnorm(dx, dr, dw, EPS)
        q = gla.add_rmsnorm_q8(dx, dr, dw, EPS)
        return [y, s, q[0].view(torch.uint8), q[1], *gla.add_rmsnorm_bwd(s, dw, EPS, dgy, gsum=dgs),
                *gla.gate_bwd(o, z, nw, EPS, gyo)]
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for i in range(3):
        dx.mul_(0.5)
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_other_stream():
    x, r, w, gy, gs = make(300, 1000, np.float32, 10)
    dx, dr, dw, dgy, dgs = to_dev(x, r, w, gy, gs)
    y, s = gla.add_rmsnorm(dx, dr, dw, EPS)
    gx, gw = gla.add_rmsnorm_bwd(s, dw, EPS, dgy)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2, s2 = gla.add_rmsnorm(dx, dr, dw, EPS, stream=st)
    gx2, gw2 = gla.add_rmsnorm_bwd(s2, dw, EPS, dgy, stream=st)
    st.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(gx, gx2) and torch.equal(gw, gw2)


def test_binding_refusals():
    x, r, w, gy, _ = make(4, 64, np.float16, 11)
    dx, dr, dw, dgy = to_dev(x, r, w, gy)
    for call in (lambda: gla.add_rmsnorm(dx, dr.float(), dw, EPS), lambda: gla.add_rmsnorm(dx, dr[:2], dw, EPS),
                 lambda: gla.add_rmsnorm(dx, dr, dw.half(), EPS), lambda: gla.add_rmsnorm(dx.t(), dr.t(), dw, EPS),
                 lambda: gla.add_rmsnorm(dx, dr, dw[:32], EPS), lambda: gla.add_rmsnorm(dx, dr, dw, EPS, out=dx.float()),
                 lambda: gla.add_rmsnorm_q8(dx, dr, dw, EPS, out=torch.empty(4, 64, dtype=torch.uint8, device="cuda")),
                 lambda: gla.add_rmsnorm_bwd(dx, dw, EPS, dgy[:3]), lambda: gla.add_rmsnorm_bwd(dx.cpu(), dw, EPS, dgy),
                 lambda: gla.gate_bwd(dx, dr, dw, EPS, dgy.float()), lambda: gla.gate_bwd(dx, dr, dw, EPS, dgy, out=(dx,)),
                 lambda: gla.add_rmsnorm(dx.bfloat16(), dr.bfloat16(), dw, EPS)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(gla.GLAError):
        gla.add_rmsnorm(dx, dr, dw, EPS, out=dx, sum_out=dx)
    with pytest.raises(gla.GLAError):
        gla.gate_bwd(dx, dr, dw, EPS, dgy, out=(dx, torch.empty_like(dx)))
    with pytest.raises(gla.GLAError):
        gla.add_rmsnorm(torch.zeros(2, 12, device="cuda"), None, torch.ones(12, device="cuda"), EPS)


def test_empty():
    e, w = torch.empty(0, 64, dtype=torch.float16, device="cuda"), torch.ones(64, device="cuda")
    y, s = gla.add_rmsnorm(e, e.clone(), w, EPS)
    assert y.shape == s.shape == (0, 64)
    gx, gw = gla.add_rmsnorm_bwd(e, w, EPS, e.clone())
    assert gx.shape == (0, 64) and not bool(gw.any())
    assert not bool(gla.gate_bwd(e, e.clone(), w, EPS, e.clone())[2].any())


def test_more_rows_than_one_launch():
    """17 million rows of 8 are two launches; the last rows against a call of
    their own, bit for bit, for both outputs; and their weight gradient."""
    rows = (1 << 24) + 777
    x = torch.zeros(rows, 8, dtype=torch.float16, device="cuda")
    r = torch.randn(rows, 8, device="cuda").half()
    w = 1 + 0.1 * torch.randn(8, device="cuda")
    x[-900:] = torch.randn(900, 8, device="cuda").half()
    y, s = gla.add_rmsnorm(x, r, w, EPS)
    y8, sc, s8 = gla.add_rmsnorm_q8(x, r, w, EPS)
    ty, ts = gla.add_rmsnorm(x[-900:], r[-900:], w, EPS)
    t8, tc, _ = gla.add_rmsnorm_q8(x[-900:], r[-900:], w, EPS)
    torch.cuda.synchronize()
    assert torch.equal(y[-900:], ty) and torch.equal(s[-900:], ts) and torch.equal(s, s8)
    assert torch.equal(y8[-900:].view(torch.uint8), t8.view(torch.uint8)) and torch.equal(sc[-900:], tc)
    g = torch.zeros_like(s)
    g[-900:] = ty
    _, gw = gla.add_rmsnorm_bwd(s, w, EPS, g)
    _, tw = gla.add_rmsnorm_bwd(ts, w, EPS, ty)
    torch.cuda.synchronize()
    # the same 900 terms in another order: 900 u of their magnitudes
    n = ts.double() / (ts.double().square().mean(1, keepdim=True) + EPS).sqrt()
    assert bool(((gw - tw).abs().double() <= 900 * U * (n * ty.double()).abs().sum(0)).all())
