"""GPU: the products and norms between a block's mixers as they are used together
(a block's training step, its tokens one by one, a channel mixer against
differences), at the borders between their forms, and what they refuse.

Bars of the runs together. Half: up to twenty tensors in a row are rounded, by
2^-11 relative each, and a branch meets the stream twice: 2% of the largest value.
Float, K <= 192: a product is off by (K + 2) 2^-23 of its sum of magnitudes, which
is below sqrt(K) times the largest output: 3e-4 for each of six products in a row,
2e-3 of the largest value with the norms and the activation."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say, to_dev
from recurrent_vision_token_gla_amd import gla
import test_gpu_gated_norm as norms
from test_gpu_linear import U, act_off, check, expect_linear, half_step, normal, sums

pytestmark = pytest.mark.gpu
EPS = 1e-6
BAR = {torch.float16: 2e-2, torch.float32: 2e-3}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def close(name, got, want, bar):
    d = (got.double().cpu() - want.detach()).abs().max().item() / want.detach().abs().max().item()
    say(f"  {name}: {d:.2e} of the largest")
    assert d <= bar, name


def rms(x, w):
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w


def channel_mixer(m, res, w, gate, scale, wg, wu, wd):
    """float64 on the CPU: (output, the stream behind the gated sum)."""
    s = res + scale * gate[:, None] * m
    y = rms(s, w)
    return s + (torch.nn.functional.silu(y @ wg.t()) * (y @ wu.t())) @ wd.t()


def channel_mixer_here(m, res, w, gate, scale, wg, wu, wd, gy):
    """The same through the library: output and the gradients of all inputs."""
    y, s = gla.gated_add_rmsnorm(m, res, w, EPS, gate=gate, scale=scale)
    h, a, u = gla.gated_ff(y, wg, wu, return_parts=True)
    out = gla.linear(h, wd, residual=s)
    ghid, gwd, _ = gla.linear_bwd(h, wd, gy, need_bias=False)
    gyn, gwg, gwu = gla.gated_ff_bwd(y, wg, wu, a, u, ghid)
    gm, gres, gw, _, ggate, gscale = gla.gated_add_rmsnorm_bwd(m, s, w, EPS, gyn, gate=gate, scale=scale, gsum=gy)
    return out, [gm, gres, gw, ggate, gscale, gwg, gwu, gwd]


def channel_mixer_inputs(B, T, F, hidden, dtype, seed):
    torch.manual_seed(seed)
    n = lambda *shape, s=1.0: (torch.randn(*shape, device="cuda") * s).to(dtype)
    return [n(B, T, F), n(B, T, F), 1 + 0.1 * torch.randn(F, device="cuda"), n(B, F),
            0.5 + 0.1 * torch.randn(F, device="cuda"), n(hidden, F, s=F ** -0.5), n(hidden, F, s=F ** -0.5),
            n(F, hidden, s=hidden ** -0.5)], n(B, T, F)


@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (2, 37), (3, 130)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_training_step_of_a_channel_mixer(B, T, dtype):
    args, gy = channel_mixer_inputs(B, T, 96, 192, dtype, B + T)
    out, grads = channel_mixer_here(*args, gy)
    torch.cuda.synchronize()
    leaves = [t.double().cpu().requires_grad_() for t in args]
    want = channel_mixer(*leaves)
    wants = torch.autograd.grad((want * gy.double().cpu()).sum(), leaves)
    close("output", out, want, BAR[dtype])
    for n, got, w in zip(["m", "residual", "norm weight", "gate", "scale", "Wg", "Wu", "Wd"], grads, wants):
        close(n, got, w, BAR[dtype])


def test_gradient_of_a_channel_mixer_against_differences():
    """Along one direction in every input: central differences of the float64
    formula, off by h^2 of a third derivative (1e-8 here)."""
    args, gy = channel_mixer_inputs(2, 9, 64, 72, torch.float32, 8)
    _, grads = channel_mixer_here(*args, gy)
    torch.cuda.synchronize()
    base, g = [t.double().cpu() for t in args], gy.double().cpu()
    for i, grad in enumerate(grads):
        d = torch.randn(base[i].shape, dtype=torch.float64)
        d /= d.norm()
        ends = []
        for h in (1e-4, -1e-4):
            moved = list(base)
            moved[i] = base[i] + h * d
            ends.append((channel_mixer(*moved) * g).sum().item())
        got = (grad.double().cpu() * d).sum().item()
        diff = (ends[0] - ends[1]) / 2e-4
        assert abs(got - diff) <= BAR[torch.float32] * grad.double().norm().item(), i


def block_weights(F, H, dk, dv, hidden):
    half = lambda *shape, s=1.0: (torch.randn(*shape, device="cuda") * s).half()
    w = dict(norm1=1 + 0.1 * torch.randn(F, device="cuda"), norm2=1 + 0.1 * torch.randn(F, device="cuda"),
             out_norm=1 + 0.1 * torch.randn(dv, device="cuda"), decay_bias=torch.randn(H * dk, device="cuda"),
             post=1 + 0.1 * torch.randn(F, device="cuda"), scale=0.5 + 0.1 * torch.randn(F, device="cuda"))
    for name, n, k in (("q", H * dk, F), ("k", H * dk, F), ("v", H * dv, F), ("g", H * dk, F), ("z", H * dv, F),
                       ("o", F, H * dv), ("gate", hidden, F), ("up", hidden, F), ("down", F, hidden)):
        w[name] = half(n, k, s=k ** -0.5)
    return w


def projections(h, w, lead, H, dk, dv):
    """q, k, v, decay and gate of the token mixer, and the decay's kept sums."""
    q = gla.linear(h, w["q"], alpha=dk ** -0.5).view(*lead, H, dk)
    k, v, z = (gla.linear(h, w[n]).view(*lead, H, d) for n, d in (("k", dk), ("v", dv), ("z", dv)))
    g, pre = gla.linear(h, w["g"], w["decay_bias"], act=gla.ACT_LOGSIGMOID, alpha=1 / 16, return_pre=True)
    return q, k, v, g.view(*lead, H, dk), z, pre


def test_training_step_of_a_block():
    """Norm, projections, recurrence with its gate, the way back into the stream
    with the post norm and scale, the gated feed-forward: forward and every
    gradient against float64 autograd."""
    torch.manual_seed(6)
    B, gh, gw, H, dk, dv, F, hidden = 2, 6, 8, 2, 32, 32, 72, 136
    T = gh * gw
    w = block_weights(F, H, dk, dv, hidden)
    half = lambda *shape: torch.randn(*shape, device="cuda").half()
    x, res, gy = half(B, T, F), half(B, T, F), half(B, T, F)
    # forward
    h1, s1 = gla.add_rmsnorm(x, res, w["norm1"], EPS)
    q, k, v, g, z, pre = projections(h1, w, (B, T), H, dk, dv)
    o = gla.fwd(q, k, v, g, gh, gw, gla.T2B)
    y = gla.fwd_gated(q, k, v, g, z, w["out_norm"], EPS, gh, gw, gla.T2B).view(B, T, -1)
    m = gla.linear(y, w["o"])
    h2, s2 = gla.gated_add_rmsnorm(m, s1, w["norm2"], EPS, post_weight=w["post"], scale=w["scale"])
    hid, a, u = gla.gated_ff(h2, w["gate"], w["up"], act=gla.ACT_GELU, return_parts=True)
    out = gla.linear(hid, w["down"], residual=s2)
    # backward
    got = {}
    ghid, got["down"], _ = gla.linear_bwd(hid, w["down"], gy, need_bias=False)
    gh2, got["gate"], got["up"] = gla.gated_ff_bwd(h2, w["gate"], w["up"], a, u, ghid, act=gla.ACT_GELU)
    gm, gs1, got["norm2"], got["post"], _, got["scale"] = gla.gated_add_rmsnorm_bwd(
        m, s2, w["norm2"], EPS, gh2, post_weight=w["post"], scale=w["scale"], gsum=gy)
    gyo, got["o"], _ = gla.linear_bwd(y, w["o"], gm, need_bias=False)
    go, gz, got["out_norm"] = gla.gate_bwd(o, z, w["out_norm"], EPS, gyo.view(B, T, H, dv))
    gq, gk, gv, gg = gla.bwd(q, k, v, g, go, gh, gw, gla.T2B)
    rows = lambda t: t.reshape(B, T, -1)
    parts = [gla.linear_bwd(h1, w["q"], rows(gq), alpha=dk ** -0.5, need_bias=False)]
    parts += [gla.linear_bwd(h1, w[n], rows(t), need_bias=False) for n, t in (("k", gk), ("v", gv), ("z", gz))]
    parts.append(gla.linear_bwd(h1, w["g"], rows(gg), act=gla.ACT_LOGSIGMOID, alpha=1 / 16, pre=pre))
    for n, p in zip("qkvzg", parts):
        got[n] = p[1]
    got["decay_bias"] = parts[-1][2]
    gh1 = sum(p[0].float() for p in parts).half()
    got["x"], got["norm1"] = gla.add_rmsnorm_bwd(s1, w["norm1"], EPS, gh1, gsum=gs1)
    torch.cuda.synchronize()

    r = {n: t.double().cpu().requires_grad_() for n, t in w.items()}
    r["x"] = x.double().cpu().requires_grad_()
    F_ = torch.nn.functional
    s = r["x"] + res.double().cpu()
    h = rms(s, r["norm1"])
    heads = lambda n, d: (h @ r[n].t()).view(B, T, H, d)
    rq, rk, rv, rz = heads("q", dk) * dk ** -0.5, heads("k", dk), heads("v", dv), heads("z", dv)
    rg = (F_.logsigmoid(h @ r["g"].t() + r["decay_bias"]) / 16).view(B, T, H, dk)
    S, ro = torch.zeros(B, H, dk, dv, dtype=torch.float64), [None] * T
    for t in torch.arange(T).view(gh, gw).t().reshape(-1).tolist():  # top to bottom
        S = S * rg[:, t].exp()[..., None] + rk[:, t][..., None] * rv[:, t][..., None, :]
        ro[t] = (rq[:, t][..., None] * S).sum(2)
    ry = rms(torch.stack(ro, 1), r["out_norm"]) * F_.silu(rz)
    s = s + r["scale"] * rms(ry.reshape(B, T, -1) @ r["o"].t(), r["post"])
    h = rms(s, r["norm2"])
    want = s + (F_.gelu(h @ r["gate"].t()) * (h @ r["up"].t())) @ r["down"].t()
    wants = torch.autograd.grad((want * gy.double().cpu()).sum(), list(r.values()))
    close("output", out, want, BAR[torch.float16])
    assert set(got) == set(r)
    for n, t in zip(r, wants):
        close(n, got[n], t, BAR[torch.float16])


def test_tokens_one_by_one_through_a_block():
    """A prompt in one go with its state handed back, then the new tokens of
    three sequences at a time, against all of it in one go."""
    torch.manual_seed(7)
    B, T0, T, H, dk, dv, F, hidden = 3, 60, 72, 2, 32, 64, 96, 264
    w = block_weights(F, H, dk, dv, hidden)
    x = torch.randn(B, T, F, device="cuda").half()
    pool = torch.zeros(B + 2, H, dk, dv, device="cuda")
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")

    def through(x, mix):
        h, s = gla.add_rmsnorm(x, None, w["norm1"], EPS)
        q, k, v, g, z, _ = projections(h, w, x.shape[:-1], H, dk, dv)
        y = mix(q, k, v, g, z)
        m = gla.linear(y.reshape(*x.shape[:-1], -1), w["o"])
        h, s = gla.gated_add_rmsnorm(m, s, w["norm2"], EPS, post_weight=w["post"], scale=w["scale"])
        return gla.linear(gla.gated_ff(h, w["gate"], w["up"]), w["down"], residual=s)

    def whole(s_final=None):
        return lambda q, k, v, g, z: gla.fwd_gated(q, k, v, g, z, w["out_norm"], EPS, 1, q.shape[1], s_final=s_final)

    def one(q, k, v, g, z):
        return gla.step_gated(q, k, v, g, z, w["out_norm"], EPS, pool, slots)

    want = through(x, whole())
    state = torch.empty(B, H, dk, dv, device="cuda")
    got = [through(x[:, :T0].contiguous(), whole(state))]
    pool[slots.long()] = state
    for t in range(T0, T):
        got.append(through(x[:, t].contiguous(), one)[:, None])
    torch.cuda.synchronize()
    close("tokens", torch.cat(got, 1), want.double().cpu(), BAR[torch.float16])


# rows and outputs around the borders between the form for few rows and the tiles
@pytest.mark.parametrize("rows", [7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65])
@pytest.mark.parametrize("N", [2048, 2056])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_borders_between_the_forms(rows, N, dtype):
    r = np.random.default_rng(rows + N)
    K = 72
    x, w, v = normal(r, dtype, rows, K), normal(r, dtype, N, K, s=K ** -0.5), normal(r, dtype, N, K, s=K ** -0.5)
    b = normal(r, np.float32, N)
    dx, dw, dv, db = to_dev(x, w, v, b)
    y, ty, pre, tpre = expect_linear(x, w, b, "gelu", 0.5, None, dtype)
    got, gpre = gla.linear(dx, dw, db, act=gla.ACT_GELU, alpha=0.5, return_pre=True)
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


def test_float_values_over_their_range():
    """Floats of 2^-100 and up to 3.3e38 through the products' terms, and what is
    not finite stays in its row, with three rows and with seventy."""
    for rows in (3, 70):
        r = np.random.default_rng(rows)
        x, w = normal(r, np.float32, rows, 40), normal(r, np.float32, 24, 40)
        for s in (2.0 ** -100, 1e38):
            # of seventy rows one holds 3.79 * 1e38, which is beyond float's largest, 3.40e38, before it is divided
            with np.errstate(over="ignore"):
                xs, ws = x * np.float32(s) / 3, w / np.float32(s)
            y = gla.linear(*to_dev(xs, ws))
            torch.cuda.synchronize()
            fin = np.isfinite(xs).all(1)
            assert fin.sum() >= rows - 1 and not torch.isfinite(y[torch.from_numpy(~fin).cuda()]).any()
            X, W = xs[fin].astype(np.float64), ws.astype(np.float64)
            S = np.abs(X) @ np.abs(W).T
            # Below 2^-110 the third term is no normal bfloat16: the smallest step is 2^-133 (2^-126 with 7 bits),
            # so an operand is kept to 2^-134. At 1e38 that is 0.4% of a weight of 1e-38, which is subnormal itself.
            low = 2.0 ** -134 * (np.abs(X).sum(1)[:, None] + np.abs(W).sum(1))
            check(f"{s:.0e}", y[torch.from_numpy(fin).cuda()], X @ W.T,
                  sums(np.float32, 40, S) + half_step(np.float32, S) + low)
        clean = gla.linear(*to_dev(x, w))
        x[1, 5], x[2, 7] = np.inf, np.nan
        got = gla.linear(*to_dev(x, w))
        torch.cuda.synchronize()
        keep = [i for i in range(rows) if i not in (1, 2)]
        assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[1:3]).any()


def test_refused_calls_leave_the_current_stream():
    s = torch.cuda.Stream()
    x, w = torch.randn(40, 32, device="cuda").half(), torch.randn(32, 32, device="cuda").half()
    n, host = torch.ones(32, device="cuda"), torch.empty(40, 32).half()
    few = torch.empty(16, dtype=torch.uint8)
    calls = [lambda: gla.linear(x, w, out=host, stream=s),
             lambda: gla.linear(x, w, return_pre=True, pre=host, stream=s),
             lambda: gla.linear_bwd(x, w, x, gx=host, stream=s),
             lambda: gla.linear_bwd(x, w, x, gbias=torch.empty(32), stream=s),
             lambda: gla.linear_bwd(x, w, x, workspace=few, stream=s),
             lambda: gla.gated_ff(x, w, w, out=host, stream=s),
             lambda: gla.gated_ff(x, w, w, return_parts=True, parts=[x, host], stream=s),
             lambda: gla.gated_ff_bwd(x, w, w, x, x, x, gx=host, stream=s),
             lambda: gla.gated_ff_bwd(x, w, w, x, x, x, workspace=few, stream=s),
             lambda: gla.gated_add_rmsnorm(x, x, n, EPS, out=host, stream=s),
             lambda: gla.gated_add_rmsnorm(x, x, n, EPS, sum_out=host, stream=s),
             lambda: gla.gated_add_rmsnorm_bwd(x, x, n, EPS, x, gx=host, stream=s),
             lambda: gla.gated_add_rmsnorm_bwd(x, x, n, EPS, x, gresidual=host, stream=s),
             lambda: gla.gated_add_rmsnorm_bwd(x, x, n, EPS, x, workspace=few, stream=s)]
    before = torch.cuda.current_stream()
    assert before != s
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
        assert torch.cuda.current_stream() == before, i
    torch.cuda.synchronize()


def test_gradients_refuse_a_prepared_workspace():
    """Memory that holds the control words of a workspace prepared for the
    forward's single pass is nobody else's."""
    x, w = torch.randn(40, 32, device="cuda").half(), torch.randn(32, 32, device="cuda").half()
    n = torch.ones(32, device="cuda")
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    gla.workspace_init(ws)
    calls = [lambda: gla.linear_bwd(x, w, x, act=gla.ACT_SILU, pre=x, workspace=ws),
             lambda: gla.gated_ff_bwd(x, w, w, x, x, x, workspace=ws),
             lambda: gla.gated_add_rmsnorm_bwd(x, x, n, EPS, x, workspace=ws)]
    for call in calls:
        with pytest.raises(gla.GLAError) as e:
            call()
        assert e.value.status == gla.E_ARG
    torch.cuda.synchronize()
    assert not bool(ws[:gla.CTRL_BYTES].any())
    gla.workspace_release(ws)
    for call in calls:
        call()
    torch.cuda.synchronize()


def test_rows_without_values_are_refused():
    """A contraction of nothing has outputs, which no call writes; without outputs
    there is nothing to do."""
    x, w = torch.empty(3, 0, device="cuda").half(), torch.empty(24, 0, device="cuda").half()
    gy = torch.zeros(3, 24, device="cuda").half()
    for call in (lambda: gla.linear(x, w), lambda: gla.gated_ff(x, w, w), lambda: gla.linear_bwd(x, w, gy),
                 lambda: gla.gated_ff_bwd(x, w, w, gy, gy, gy)):
        with pytest.raises(gla.GLAError) as e:
            call()
        assert e.value.status == gla.E_UNSUPPORTED
    assert gla.linear(x, w[:0]).shape == (3, 0)
    y, s = gla.gated_add_rmsnorm(x, x, torch.empty(0, device="cuda"), EPS)
    assert y.shape == s.shape == (3, 0)


def test_many_rows_and_offsets_beyond_32_bits():
    """More rows than one launch takes, outputs of more than 4 GiB. Values are
    whole and small, so that every sum is exact in float."""
    rows, K, N = (1 << 22) + 17, 8, 520
    torch.manual_seed(9)
    whole = lambda *shape: torch.randint(-1, 2, shape, device="cuda", dtype=torch.int8).half()
    x, w = whole(rows, K), whole(N, K)
    y = gla.linear(x, w)
    h, a, u = gla.gated_ff(x, w, w, act=gla.ACT_NONE, return_parts=True)
    torch.cuda.synchronize()
    some = torch.cat([torch.arange(70), torch.arange((1 << 22) - 40, rows), torch.arange(1 << 21, (1 << 21) + 70)]).cuda()
    want = x[some].float() @ w.float().t()
    for got, t in ((y, want), (a, want), (u, want), (h, want * want)):
        assert torch.equal(got[some].float(), t)
    del y, a, u
    gy = h.clamp_(-1, 1)
    gx, gw, gb = gla.linear_bwd(x, w, gy)
    torch.cuda.synchronize()
    assert torch.equal(gx[some].float(), gy[some].float() @ w.float())
    gW, gB = torch.zeros(N, K, device="cuda"), torch.zeros(N, device="cuda")
    for r in range(0, rows, 1 << 19):
        g = gy[r:r + (1 << 19)].float()
        gW += g.t() @ x[r:r + (1 << 19)].float()
        gB += g.sum(0)
    assert gW.abs().max() < 1 << 24 and gB.abs().max() < 1 << 24
    assert torch.equal(gw, gW.half()) and torch.equal(gb, gB)
    del x, h, gy, gx
    torch.cuda.empty_cache()


def test_norms_with_offsets_beyond_32_bits():
    rows, F, G = (1 << 21) + 2, 1032, 2
    torch.manual_seed(10)
    x, res = (torch.randn(rows, F, device="cuda", dtype=torch.float16) for _ in range(2))
    w, gate = torch.ones(F, device="cuda"), torch.randn(G, F, device="cuda").half()
    y, s = gla.gated_add_rmsnorm(x, res, w, EPS, gate=gate)
    gx, gres, _, _, ggate, _ = gla.gated_add_rmsnorm_bwd(x, s, w, EPS, res, gate=gate)
    torch.cuda.synchronize()
    for r in (slice(0, 50), slice(rows // 2 - 50, rows // 2), slice(rows // 2, rows // 2 + 50), slice(rows - 50, rows)):
        g = gate[r.start * G // rows][None].contiguous()
        part = gla.gated_add_rmsnorm(x[r], res[r], w, EPS, gate=g)
        back = gla.gated_add_rmsnorm_bwd(x[r], part[1], w, EPS, res[r], gate=g)
        torch.cuda.synchronize()
        for got, want in zip((y, s, gx, gres), (*part, *back[:2])):
            assert torch.equal(got[r], want)
    del x, res, y, s, gx, gres, got
    torch.cuda.empty_cache()


# groups of a gate's rows around the ways their sums are shared out: a team or a workgroup to a group, one
# or several workgroups, more groups than the last launch takes side by side
@pytest.mark.parametrize("G,per,F", [(8, 5, 40), (9, 5, 40), (20, 70, 64), (300, 3, 72), (511, 2, 24), (512, 6, 40),
                                     (600, 7, 72), (600, 8, 72), (520, 12, 264), (1100, 2, 1032), (9, 300, 64)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_norms_with_groups_of_every_number(G, per, F, dtype):
    norms.test_forward(G, per, F, dtype)
    for carry in (True, False):
        norms.test_backward(G, per, F, dtype, carry)
