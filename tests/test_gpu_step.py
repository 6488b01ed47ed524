"""GPU: the recurrence for one new token per row on a pool of states
(gla_step, gla_step_gated) against the float64 recurrence.

Tolerance, in units u = 2^-24. State: one product and one fused addition after
a decay that is off by at most (2 + |gk log2 e|) u (its argument is rounded
once): (4 + 2 |gk|) u of the terms' magnitudes. Output: 64 of those summed, 64
u more of sum |q S|, and half a step of the type. Gated: the norm and the gate
multiply o by factors that are off by at most 8 u, and rows near zero divide
o's error by their own size: the bound follows the error through
y = o r w silu(z), |dy| <= (|do| + |o| sum|o do| r^2 / dv) r |w silu(z)|."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def make(B, H, dk, dv, n, dtype, seed):
    r = np.random.default_rng(seed)
    q = r.standard_normal((B, H, dk)) * dk ** -0.5
    k, g = r.standard_normal((B, H, dk)), -np.exp(r.uniform(-6, 1, (B, H, dk)))
    v, z = r.standard_normal((B, H, dv)), r.standard_normal((B, H, dv))
    return ([a.astype(dtype) for a in (q, k, v, g)], z.astype(dtype),
            (1 + 0.1 * r.standard_normal(dv)).astype(np.float32),
            r.standard_normal((n, H, dk, dv)).astype(np.float32))


def reference(x, z, w, state, slots, gated):
    """Row by row in row order: outputs and states with the bound of each."""
    q, k, v, g = (a.astype(np.float64) for a in x)
    S, dS = state.astype(np.float64), np.zeros(state.shape)
    B, H, _ = q.shape
    out, tol = np.full(v.shape, np.nan), np.zeros(v.shape)
    half = 2.0 ** -11 if x[0].dtype == np.float16 else U
    for b, s in enumerate(slots):
        if s < 0 or s >= len(S):
            continue
        a = np.exp(g[b])[..., None]
        kv = k[b][..., None] * v[b][:, None, :]
        mag = a * np.abs(S[s]) + np.abs(kv)
        dS[s] = a * dS[s] + (4 + 2 * np.abs(g[b][..., None])) * U * mag
        S[s] = a * S[s] + kv
        o = np.einsum("hd,hde->he", q[b], S[s])
        do = np.einsum("hd,hde->he", np.abs(q[b]), dS[s] + 64 * U * np.abs(S[s]))
        if gated:
            r = 1 / np.sqrt(np.mean(o * o, -1, keepdims=True) + EPS)
            f = np.abs(w * oracle.silu(z[b]))
            do = (do + np.abs(o) * np.mean(np.abs(o) * do, -1, keepdims=True) * r ** 2 * 2 + 16 * U * np.abs(o)) * r * f
            o = oracle.rmsnorm_gate(o, z[b], w, EPS)
        out[b], tol[b] = o, do + half * np.abs(o) + (2.0 ** -25 if half > U else 0)
    return out, tol, S, dS + U * np.abs(S)


def run(x, z, w, state, slots, gated, out=None, **kw):
    dev, ds = to_dev(*x), to_dev(state)[0]
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    if gated:
        y = gla.step_gated(*dev, *to_dev(z, w), EPS, ds, sl, out=out, **kw)
    else:
        y = gla.step(*dev, ds, sl, out=out, **kw)
    torch.cuda.synchronize()
    return y.double().cpu().numpy(), ds.double().cpu().numpy()


def check(B, H, dk, dv, n, dtype, slots, gated, seed):
    x, z, w, state = make(B, H, dk, dv, n, dtype, seed)
    rows = list(range(B)) if slots is None else slots
    want, tol, S, dS = reference(x, z, w, state, rows, gated)
    out = torch.full((B, H, dv), 7.0, dtype=torch.float16 if dtype == np.float16 else torch.float32, device="cuda")
    got, gS = run(x, z, w, state, slots, gated, out=out)
    skipped = np.isnan(want)
    assert np.all(got[skipped] == 7)  # padding rows are left as they were
    worst = float(np.max(np.abs(got - want)[~skipped] / tol[~skipped])) if (~skipped).any() else 0.0
    ws = float(np.max(np.abs(gS - S) / np.maximum(dS, 1e-30)))
    say(f"step B={B} H={H} {dk}/{dv} n={n} {np.dtype(dtype).name} gated={gated}: out {worst:.3f}, state {ws:.3f} of the bound")
    assert worst <= 1 and ws <= 1
    untouched = [s for s in range(n) if s not in rows]
    assert np.array_equal(gS[untouched], state.astype(np.float64)[untouched])


@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 64), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("gated", [False, True])
def test_shapes(dk, dv, dtype, gated):
    check(3, 5, dk, dv, 3, dtype, None, gated, 10 + dk + dv)
    check(5, 3, dk, dv, 9, dtype, [8, 0, 3, 7, 1], gated, 20 + dk + dv)


@pytest.mark.parametrize("gated", [False, True])
def test_padding_rows(gated):
    check(6, 2, 64, 64, 4, np.float16, [2, -1, 0, 4, 2 ** 31 - 1, 3], gated, 40)
    check(3, 2, 64, 64, 2, np.float16, [-1, -5, -(2 ** 31)], gated, 41)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_of_one_slot_apply_in_order(dtype, gated):
    check(7, 2, 64, 64, 3, dtype, [1, 0, 1, 1, 2, 0, 1], gated, 50)
    # a whole sequence in one call, among others, over several groups of 64 rows
    r = np.random.default_rng(5)
    check(200, 1, 32, 64, 4, dtype, [int(s) for s in r.integers(-1, 4, 200)], gated, 51)


def test_one_row_and_many():
    # more rows than one round of slot comparisons, slots shared far apart
    r = np.random.default_rng(8)
    check(1200, 1, 32, 32, 500, np.float16, [int(s) for s in r.integers(-1, 500, 1200)], False, 62)
    check(1, 1, 64, 64, 1, np.float16, None, False, 60)
    check(300, 3, 32, 32, 400, np.float16, [int(s) for s in np.random.default_rng(6).permutation(400)[:300]], True, 61)


def test_tokens_one_by_one_equal_the_whole_sequence():
    """Serving a sequence through gla_step gives what gla_fwd_state gives for
    it at once, within the forward's bar, and the same final state."""
    T, H, dk, dv = 70, 3, 64, 64
    r = np.random.default_rng(7)
    q, k, v, g = (r.standard_normal((2, T, H, d)).astype(np.float16) for d in (dk, dk, dv, dk))
    q, g = (q * np.float16(0.125)), -np.abs(g) / 16
    dev = to_dev(q, k, v, g)
    o, sT = gla.fwd_state(*dev, 1, T, 0)
    pool = torch.zeros(5, H, dk, dv, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    steps = torch.stack([gla.step(*[t[:, i].contiguous() for t in dev], pool, slots) for i in range(T)], 1)
    torch.cuda.synchronize()
    assert float((steps.double() - o.double()).abs().max() / o.double().abs().max()) <= 5e-3
    assert float((pool[slots.long()] - sT).abs().max() / sT.abs().max()) <= 5e-3


def test_graph_replays_advance_the_states():
    x, z, w, state = make(4, 2, 64, 64, 6, np.float16, 70)
    dev, ds = to_dev(*x), to_dev(state)[0]
    slots = torch.tensor([5, -1, 0, 5], dtype=torch.int32, device="cuda")
    dz, dw = to_dev(z, w)
    out = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    ref, rout = ds.clone(), out.clone()
    gla.step_gated(*dev, dz, dw, EPS, ref, slots, out=rout)
    torch.cuda.synchronize()
    ref.copy_(ds)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gla.step_gated(*dev, dz, dw, EPS, ds, slots, out=out)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        gla.step_gated(*dev, dz, dw, EPS, ref, slots, out=rout)
        torch.cuda.synchronize()
        assert torch.equal(ds, ref) and torch.equal(out, rout)


def test_other_stream():
    x, z, w, state = make(8, 4, 64, 64, 8, np.float16, 71)
    want, S = run(x, z, w, state, None, False)
    s = torch.cuda.Stream()
    dev, ds = to_dev(*x), to_dev(state)[0]
    s.wait_stream(torch.cuda.current_stream())
    y = gla.step(*dev, ds, stream=s)
    s.synchronize()
    assert np.array_equal(y.double().cpu().numpy(), want) and np.array_equal(ds.double().cpu().numpy(), S)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: its last slot."""
    n, H, dk, dv = 70000, 4, 64, 64  # 4.6e9 bytes, 1.1e9 floats
    pool = torch.zeros(n, H, dk, dv, device="cuda")
    x, _, _, _ = make(2, H, dk, dv, 1, np.float16, 72)
    dev = to_dev(*x)
    small = torch.zeros(2, H, dk, dv, device="cuda")
    want = gla.step(*dev, small)
    got = gla.step(*dev, pool, torch.tensor([n - 1, n // 2], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(pool[[n - 1, n // 2]], small)
    pool[[n - 1, n // 2]] = 0
    assert not bool(pool.any())


def test_binding_refusals():
    x, z, w, state = make(2, 2, 32, 64, 3, np.float16, 73)
    q, k, v, g = to_dev(*x)
    ds = to_dev(state)[0]
    bad = [lambda: gla.step(q, k, v, g, ds.half()), lambda: gla.step(q, k, v[:, :, :32], g, ds),
           lambda: gla.step(q[:, :, ::2], k, v, g, ds), lambda: gla.step(q, k, v, g, ds[:1]),
           lambda: gla.step(q, k, v, g, ds, torch.tensor([0, 1], device="cuda")),
           lambda: gla.step(q, k, v, g, ds, torch.tensor([0], dtype=torch.int32, device="cuda")),
           lambda: gla.step(q, k, v, g, ds, torch.tensor([0, 1], dtype=torch.int32)),
           lambda: gla.step(q.float(), k, v, g, ds), lambda: gla.step(q, k, v, g, ds.transpose(2, 3)),
           lambda: gla.step_gated(q, k, v, g, v.float(), to_dev(w)[0], EPS, ds)]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(gla.GLAError):
        gla.step(q, k, v, g, ds, out=v)
    empty = torch.empty(0, 2, 32, dtype=torch.float16, device="cuda")
    assert gla.step(empty, empty, torch.empty(0, 2, 64, dtype=torch.float16, device="cuda"), empty, ds).shape == (0, 2, 64)
