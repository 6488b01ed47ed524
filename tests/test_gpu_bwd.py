"""GPU: gradients of the recurrence (gla_bwd) against the float64 oracle.

Tolerance. Let M be what the formula gives when every term is taken in
magnitude (the oracle on |q|, |k|, |v|, |go|, |s0|, |gs_final| with the same
decays). In units u = 2^-24 of M an output may be off by
  * operands: half inputs are carried in two bf16 terms, each operand off by at
    most 2^-18 and the product of the two second terms (2^-18) left out, over
    at most two chained products and a carried state: 8 * 2^-18 = 512 u; float
    inputs in three terms, 2^-27 each and 2^-26 left out: at most 8 * 2^-25 = 4 u;
  * sums: a product sums 64 elements, at most three of them chained: 192 u; the
    states sum over N chunks: N u;
  * decays: exponents are sums of decays whose magnitude stays below G = the
    largest |log2 decay| summed over a 16-token block (160 per token at most),
    each sum off by 8 G u, times ln 2: 6 G u;
plus half a step of the output type, eps/2 of the value (and half the smallest
subnormal of half). The decay's gradient also takes differences inside a chunk:
its M adds twice the chunk's sum of |q| M_gq over the tokens behind."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from oracle import to_raster, to_scan
from recurrent_vision_token_gla_amd import gla
from recurrent_vision_token_gla_amd import workloads as W

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def inputs(B, gh, gw, H, dk, dv, dtype, seed, gate="plain", carry=False, gate_override=None):
    x = W.make_inputs(B, gh * gw, H, dk, dv, dtype, seed=seed, gate=gate, gate_override=gate_override)
    rng = np.random.default_rng(seed + 5000)
    go = rng.standard_normal((B, gh * gw, H, dv)).astype(dtype)
    s0 = rng.standard_normal((B, H, dk, dv)).astype(np.float32) if carry else None
    gsf = rng.standard_normal((B, H, dk, dv)).astype(np.float32) if carry else None
    return x + (go,), s0, gsf


def bounds(x, gh, gw, dirs, s0, gsf, grads):
    """How far each output may be off, as the module's docstring derives."""
    q, k, v, g, go = x
    mag = lambda a: None if a is None else np.abs(a.astype(np.float64))
    M = list(oracle.gla_backward(mag(q), mag(k), mag(v), g, mag(go), gh, gw, dirs, mag(s0), mag(gsf)))
    B, T, H, dk = q.shape
    N = -(-T // 64)
    z = to_scan(mag(q) * M[0], gh, gw, dirs)
    z = np.pad(z, ((0, 0), (0, N * 64 - T), (0, 0), (0, 0))).reshape(B, N, 64, H, dk)
    behind = np.flip(np.cumsum(np.flip(z, 2), 2), 2).reshape(B, N * 64, H, dk)[:, :T]
    M[3] = M[3] + 2 * to_raster(np.ascontiguousarray(behind), gh, gw, dirs)
    g2 = to_scan(np.minimum(np.abs(g.astype(np.float64)) * np.log2(np.e), 160), gh, gw, dirs)
    n16 = -(-T // 16)
    G = np.pad(g2, ((0, 0), (0, n16 * 16 - T), (0, 0), (0, 0))).reshape(B, n16, 16, H, dk).sum(2).max()
    half = x[0].dtype == np.float16
    c = ((512 if half else 4) + 192 + N + 6 * G) * U
    out = [c * m + (2.0 ** -11 if half else U) * np.abs(r) + (2.0 ** -25 if half else 1e-37)
           for m, r in zip(M[:4], grads[:4])]
    return out + [c * M[4] + U * np.abs(grads[4]) + 1e-37]


def run(x, gh, gw, dirs, s0=None, gsf=None, gs0=True, **kw):
    dev = to_dev(*x)
    ds0, dgs = (None if a is None else to_dev(a)[0] for a in (s0, gsf))
    r = gla.bwd(*dev, gh, gw, list(dirs), s0=ds0, gs_final=dgs, return_gs0=gs0, **kw)
    torch.cuda.synchronize()
    return [t.double().cpu().numpy() for t in r]


def check(x, gh, gw, dirs, s0=None, gsf=None):
    ref = oracle.gla_backward(*x, gh, gw, dirs, s0, gsf)
    tol = bounds(x, gh, gw, dirs, s0, gsf, ref)
    got = run(x, gh, gw, dirs, s0, gsf)
    for n, a, r, t in zip(("gq", "gkey", "gv", "ggk", "gs0"), got, ref, tol):
        worst = float(np.max(np.abs(a - r) / t))
        say(f"  {n}: {worst:.3f} of the bound, rel {np.linalg.norm(a - r) / max(1e-300, np.linalg.norm(r)):.1e}")
        assert worst <= 1, n
    return got


@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 64), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("carry", [False, True])
def test_shapes(dk, dv, dtype, carry):
    gh, gw, dirs = 9, 17, (1, 2)
    say(f"bwd dk={dk} dv={dv} {np.dtype(dtype).name} carry={carry}")
    x, s0, gsf = inputs(2, gh, gw, 3, dk, dv, dtype, 900 + dk + dv, carry=carry)
    check(x, gh, gw, dirs, s0, gsf)


@pytest.mark.parametrize("gh,gw", [(1, 1), (1, 2), (3, 5), (4, 4), (1, 17), (7, 9), (8, 8), (5, 13), (1, 129)])
@pytest.mark.parametrize("direction", [0, 1, 2, 3])
def test_lengths_and_directions(gh, gw, direction):
    say(f"bwd grid={gh}x{gw} dir={direction}")
    x, s0, gsf = inputs(1, gh, gw, 2, 64, 64, np.float16, 920 + gh * gw, carry=True)
    check(x, gh, gw, (direction,), s0, gsf)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("gate", ["mixed", "zero", "strong", "cliff", "lowest", "random"])
def test_decays(gate, dtype):
    """Channels that keep, that forget at once, a single token that forgets
    everything, the type's lowest value, and decays from weak to strong: the
    sub-blocks with a reference and those that sum their pairs directly."""
    gh, gw, B, H, dk, dv = 10, 13, 1, 2, 64, 64
    rng = np.random.default_rng(31)
    shape = (B, gh * gw, H, dk)
    g = {"zero": np.zeros(shape), "strong": np.full(shape, -6.0) - rng.random(shape),
         "cliff": np.where(rng.random(shape) < 0.05, -60.0, -0.01),
         "lowest": np.where(rng.random(shape) < 0.1, np.finfo(dtype).min, -0.1),
         "random": -np.exp(rng.uniform(-8, 4, shape))}.get(gate)
    say(f"bwd gate={gate} {np.dtype(dtype).name}")
    x, s0, gsf = inputs(B, gh, gw, H, dk, dv, dtype, 940, gate="mixed" if g is None else "plain",
                        carry=True, gate_override=g)
    check(x, gh, gw, (3,), s0, gsf)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_large_and_small_values(dtype):
    """Values at the contract's limit, and gradients far below one."""
    gh, gw = 6, 12
    x, s0, gsf = inputs(1, gh, gw, 2, 32, 64, np.float32, 950, carry=True)
    q, k, v, g, go = x
    big = lambda a: np.clip(a * 20000, -65504, 65504)
    for name, y in (("large", (big(q) / 64, big(k) / 64, v, g, go * 0.01)), ("small", (q, k, v, g, go * 1e-4))):
        say(f"bwd {name} {np.dtype(dtype).name}")
        y = tuple(a.astype(dtype) for a in y)
        if name == "large" and dtype == np.float16:
            continue  # the outputs leave the half range
        check(y, gh, gw, (0,), s0, gsf)


@pytest.mark.parametrize("wi,direction", [(1, 1), (2, 2)])
def test_workload_shapes(wi, direction):
    w = W.WORKLOADS[wi]
    say(f"bwd {w.name}")
    x, _, _ = inputs(w.B, w.grid_h, w.grid_w, 2, w.dk, w.dv, np.float16, 960 + wi, gate="mixed")
    check(x, w.grid_h, w.grid_w, (direction,))


def test_long_ragged_sequence_float():
    x, s0, gsf = inputs(1, 1, 4099, 2, 32, 64, np.float32, 970, carry=True)
    check(x, 1, 4099, (0,), s0, gsf)


@pytest.mark.parametrize("seed", range(12))
def test_random_cases(seed):
    rng = np.random.default_rng(7000 + seed)
    B, H = int(rng.integers(1, 4)), int(rng.integers(1, 5))
    gh, gw = (int(rng.integers(1, 24)) for _ in range(2))
    dk, dv = (int(rng.choice([32, 64])) for _ in range(2))
    dtype = [np.float16, np.float32][int(rng.integers(2))]
    dirs = [int(d) for d in rng.integers(0, 4, B)]
    gate = ["plain", "mixed"][int(rng.integers(2))]
    carry = bool(rng.integers(2))
    say(f"bwd seed={seed} B={B} H={H} {gh}x{gw} {dk}/{dv} {np.dtype(dtype).name} {gate} dirs={dirs} carry={carry}")
    x, s0, gsf = inputs(B, gh, gw, H, dk, dv, dtype, 7100 + seed, gate=gate, carry=carry)
    check(x, gh, gw, dirs, s0, gsf)


def test_more_batch_elements_than_one_launch():
    """1,027 batch elements are two launches; each of the second's is right."""
    x, _, _ = inputs(1027, 1, 5, 1, 32, 32, np.float16, 980)
    dirs = [b % 4 for b in range(1027)]
    check(x, 1, 5, dirs)


def test_many_chains_take_the_serial_scan():
    """60 chains of 64/64 are 61,440 groups of four state elements: the scan
    that walks each chain in order; ten chunks, whole windows and a rest."""
    x, s0, gsf = inputs(4, 25, 25, 15, 64, 64, np.float16, 981, gate="mixed", carry=True)
    check(x, 25, 25, [0, 1, 2, 3], s0, gsf)


def test_more_chunks_than_one_window_of_the_scan():
    """131 chunks: one whole window of 16 segments of eight, and a rest that
    leaves most of the segments empty."""
    x, s0, gsf = inputs(1, 43, 195, 2, 32, 32, np.float16, 983, gate="mixed", carry=True)
    check(x, 43, 195, (2,), s0, gsf)


def test_prepared_workspace_is_refused():
    """A workspace prepared for the forward keeps control words that a gradient
    would overwrite: refused, and the forward still runs in it."""
    x, _, _ = inputs(1, 8, 24, 2, 64, 64, np.float16, 985)
    d = [torch.from_numpy(a).cuda() for a in x]
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    gla.workspace_init(ws)
    want = gla.fwd(*d[:4], 8, 24, 0, workspace=ws)
    with pytest.raises(gla.GLAError) as e:
        gla.bwd(*d, 8, 24, 0, workspace=ws)
    assert e.value.status == gla.E_ARG
    assert torch.equal(gla.fwd(*d[:4], 8, 24, 0, workspace=ws), want)
    gla.workspace_release(ws)
    for a, b in zip(gla.bwd(*d, 8, 24, 0, workspace=ws), gla.bwd(*d, 8, 24, 0)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """33.6 million token-heads: tensors of more than 2^31 elements. The last
    batch element against a call of its own, bit for bit."""
    B, H, gh, gw = 41, 16, 200, 256
    rng = torch.Generator(device="cuda").manual_seed(5)
    one = [torch.randn(1, gh * gw, H, 64, generator=rng, device="cuda").half() for _ in range(5)]
    one[3] = -one[3].abs() / 8
    big = [torch.zeros(B, gh * gw, H, 64, dtype=torch.float16, device="cuda") for _ in one]
    for t, o in zip(big, one):
        t[B - 1:] = o
    want = gla.bwd(*one, gh, gw, 2)
    got = gla.bwd(*big, gh, gw, 2)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[B - 1:], b) and not bool(a[:B - 1].any())


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_gradient_matches_differences(dtype):
    """Central differences of the float64 recurrence along random directions of
    signs, step h = 1e-5. The difference of a path of n <= 66 tokens is off by
    (n h)^2 / 6 < 1e-7 of itself, and by float64's rounding over the step,
    1e-16 / 1e-5 of the loss's terms; the gradient by the module's bounds,
    summed over the direction. (The GPU's own forward cannot be differenced
    finely: it rounds its operands to half.)"""
    gh, gw, dirs = 6, 11, [2]
    x, s0, gsf = inputs(1, gh, gw, 2, 32, 32, dtype, 990, carry=True)
    ref = oracle.gla_backward(*x, gh, gw, dirs, s0, gsf)
    tol = bounds(x, gh, gw, dirs, s0, gsf, ref)
    grads = run(x, gh, gw, dirs, s0, gsf)
    y = [a.astype(np.float64) for a in x] + [s0.astype(np.float64)]
    rng = np.random.default_rng(3)
    h = 1e-5
    for i, j in ((0, 0), (1, 1), (2, 2), (3, 3), (5, 4)):
        d = rng.choice([-1.0, 1.0], y[i].shape)

        def loss(sign):
            z = list(y)
            z[i] = y[i] + sign * h * d
            o, sT = oracle.gla_forward(*z[:4], gh, gw, dirs, s0=z[5], return_state=True)
            return np.sum(o * y[4]) + np.sum(sT * gsf)
        want, got = (loss(1) - loss(-1)) / (2 * h), float(np.sum(grads[j] * d))
        allowed = float(np.sum(tol[j])) + 1e-6 * float(np.sum(np.abs(grads[j])))
        say(f"  input {i}: derivative {got:.5f}, difference {want:.5f}, bound {allowed:.5f}")
        assert abs(got - want) <= allowed


def test_in_place_state_gradient_and_given_outputs():
    gh, gw, dirs = 8, 10, [0, 3]
    x, s0, gsf = inputs(2, gh, gw, 2, 64, 32, np.float16, 991, carry=True)
    want = run(x, gh, gw, dirs, s0, gsf)
    dev, ds0, dgs = to_dev(*x), to_dev(s0)[0], to_dev(gsf)[0]
    outs = tuple(torch.full_like(t, float("nan")) for t in dev[:4])
    ws = torch.full((gla.bwd_workspace_bytes(2, 2, gh, gw, 64, 32),), 0xFF, dtype=torch.uint8, device="cuda")
    r = gla.bwd(*dev, gh, gw, dirs, s0=ds0, gs_final=dgs, return_gs0=True, gs0=dgs, out=outs, workspace=ws)
    torch.cuda.synchronize()
    assert r[4] is dgs and all(a is b for a, b in zip(r, outs))
    for a, b in zip(r, want):
        assert np.array_equal(a.double().cpu().numpy(), b)  # any workspace contents, same bits


def test_nothing_outside_the_outputs_is_written():
    gh, gw = 5, 15
    x, s0, gsf = inputs(1, gh, gw, 3, 32, 64, np.float16, 992, carry=True)
    dev = to_dev(*x)
    frames = [torch.full((t.numel() + 128,), 7.0, dtype=t.dtype, device="cuda") for t in dev[:4]]
    outs = [f[64:-64].view(t.shape) for f, t in zip(frames, dev)]
    need = gla.bwd_workspace_bytes(1, 3, gh, gw, 32, 64)
    wsf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    gla.bwd(*dev, gh, gw, 1, out=outs, workspace=wsf[256:-256])
    torch.cuda.synchronize()
    for f in frames:
        assert bool((f[:64] == 7).all()) and bool((f[-64:] == 7).all())
    assert bool((wsf[:256] == 0x5A).all()) and bool((wsf[-256:] == 0x5A).all())


def test_non_finite_inputs_stay_in_their_chunk():
    """A NaN in a later chunk's go leaves the earlier outputs that do not
    depend on it alone: gv, gkey and ggk of an earlier token do depend on later
    go, gq does not, nor does another head."""
    x, _, _ = inputs(1, 1, 200, 2, 32, 32, np.float16, 993)
    clean = run(x, 1, 200, [0], gs0=False)
    x[4][0, 150, 1, 3] = np.nan
    got = run(x, 1, 200, [0], gs0=False)
    for a, b in zip(got, clean):
        assert np.array_equal(a[:, :, 0], b[:, :, 0])
    assert np.array_equal(got[0][:, :128, 1], clean[0][:, :128, 1])
    assert np.isnan(got[0][0, 150, 1]).all()


def test_graph_replays_with_eager_work_between():
    gh, gw, dirs = 12, 12, [1, 2]
    x, s0, gsf = inputs(2, gh, gw, 2, 64, 64, np.float16, 994, carry=True)
    dev, ds0, dgs = to_dev(*x), to_dev(s0)[0], to_dev(gsf)[0]
    outs = [torch.empty_like(t) for t in dev[:4]]
    g0 = torch.empty_like(ds0)
    ws = torch.empty(gla.bwd_workspace_bytes(2, 2, gh, gw, 64, 64), dtype=torch.uint8, device="cuda")
    call = lambda: gla.bwd(*dev, gh, gw, dirs, s0=ds0, gs_final=dgs, return_gs0=True, gs0=g0, out=outs, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    other, _, _ = inputs(2, gh, gw, 2, 64, 64, np.float16, 995)
    for new in (x, other, x):
        for t, a in zip(dev, new):
            t.copy_(torch.from_numpy(a))
        want = [t.clone() for t in gla.bwd(*dev, gh, gw, dirs, s0=ds0, gs_final=dgs, return_gs0=True)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(list(outs) + [g0], want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    gh, gw = 16, 16
    cases = [inputs(1, gh, gw, 4, 64, 64, np.float16, 996 + i, gate="mixed")[0] for i in range(2)]
    want = [run(c, gh, gw, [i], gs0=False) for i, c in enumerate(cases)]
    dev = [to_dev(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got = [gla.bwd(*d, gh, gw, i, stream=s) for i, (d, s) in enumerate(zip(dev, streams))]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert np.array_equal(a.double().cpu().numpy(), b)


def test_binding_refusals():
    x, s0, _ = inputs(1, 4, 5, 2, 32, 64, np.float16, 998, carry=True)
    q, k, v, g, go = to_dev(*x)
    ds0 = to_dev(s0)[0]
    with pytest.raises(ValueError):
        gla.bwd(q, k, v, g, go.float(), 4, 5)
    with pytest.raises(ValueError):
        gla.bwd(q, k, v, g, go[:, :, :, :32], 4, 5)
    with pytest.raises(ValueError):
        gla.bwd(q, k, v, g, go, 4, 6)
    with pytest.raises(ValueError):
        gla.bwd(q, k, v, g, go, 4, 5, gs0=ds0)                       # without return_gs0
    with pytest.raises(ValueError):
        gla.bwd(q, k, v, g, go, 4, 5, s0=ds0.half())
    with pytest.raises(ValueError):
        gla.bwd(q, k, v, g, go, 4, 5, out=(q, k, v))
    with pytest.raises(gla.GLAError):
        gla.bwd(q, k, v, g, go, 4, 5, out=(q, *[torch.empty_like(t) for t in (k, v, g)]))  # over an input
    with pytest.raises(gla.GLAError):
        gla.bwd(q, k, v, g, go, 4, 5, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gla.bwd(q.transpose(1, 2), k, v, g, go, 4, 5)


def test_empty():
    z = lambda *s: torch.empty(*s, dtype=torch.float16, device="cuda")
    r = gla.bwd(z(0, 20, 2, 32), z(0, 20, 2, 32), z(0, 20, 2, 64), z(0, 20, 2, 32), z(0, 20, 2, 64), 4, 5, [])
    assert [tuple(t.shape) for t in r] == [(0, 20, 2, 32)] * 2 + [(0, 20, 2, 64), (0, 20, 2, 32)]
    gsf = torch.randn(1, 2, 32, 64, device="cuda")
    r = gla.bwd(z(1, 0, 2, 32), z(1, 0, 2, 32), z(1, 0, 2, 64), z(1, 0, 2, 32), z(1, 0, 2, 64), 0, 5,
                gs_final=gsf, return_gs0=True)
    assert torch.equal(r[4], gsf)
