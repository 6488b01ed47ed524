"""Cases of the products and norms between a block's mixers, each in a plain
form (elementary torch operations) and as the calls a user makes.

op "linear"     y = alpha * act(x W^T + bias) + residual
op "linearbwd"  its gradient: gx, gweight, gbias
op "ff"         gated feed-forward h = act(x Wg^T) * (x Wu^T), for training
                with x Wg^T and x Wu^T kept
op "ffbwd"      its gradient: gx and both weights'
op "norm2"      norms after and before a block, its gate and residual scale:
                s = residual + scale * gate * RMSNorm(x) * post, y = RMSNorm(s) * w
op "norm2bwd"   its gradient

`own` chooses between the two forms; prepare() makes the same inputs for both.
"""
import math

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one stream: q, k, v, decay and gate projections of a 768-wide block in one
        dict(name="linear_1x768x3840", op="linear", rows=1, K=768, N=3840, dtype="f16", act="none",
             bias=True, residual=False, alpha=1.0, pre=False),
        # the channel mixer's way back into the stream, four 1280x1280 images
        dict(name="linear_25600x2048x768_res", op="linear", rows=25600, K=2048, N=768, dtype="f16",
             act="none", bias=False, residual=True, alpha=1.0, pre=False),
        # training the decay projection of one 640x640 image (12 heads of 64), latency counts
        dict(name="linearbwd_1600x768x768_logsigmoid", op="linearbwd", rows=1600, K=768, N=768,
             dtype="f16", act="logsigmoid", bias=True, alpha=1 / 16),
        # float32, odd rows and widths
        dict(name="linearbwd_1601x1000x520_gelu_f32", op="linearbwd", rows=1601, K=1000, N=520,
             dtype="f32", act="gelu", bias=True, alpha=1.0),
        # serving: the channel mixer of 37 streams' next tokens
        dict(name="ff_37x768x2048", op="ff", rows=37, K=768, F=2048, dtype="f16", act="silu", parts=False),
        # training: four 1280x1280 images, both projections kept for the gradient
        dict(name="ff_25600x768x2048_parts", op="ff", rows=25600, K=768, F=2048, dtype="f16", act="silu",
             parts=True),
        # its gradient
        dict(name="ffbwd_25600x768x2048", op="ffbwd", rows=25600, K=768, F=2048, dtype="f16", act="silu"),
        # a short ragged batch in float32
        dict(name="ffbwd_421x384x1032_f32", op="ffbwd", rows=421, K=384, F=1032, dtype="f32", act="gelu"),
        # between two mixers of one 640x640 image, a layer scale and no gate
        dict(name="norm2_1600x768", op="norm2", groups=1, per=1600, F=768, dtype="f16", post=True,
             gate=False, scale=True),
        # four 1280x1280 images, each with its own gate
        dict(name="norm2_4x6400x768_gate", op="norm2", groups=4, per=6400, F=768, dtype="f16", post=True,
             gate=True, scale=True),
        # training the same
        dict(name="norm2bwd_4x6400x768_gate", op="norm2bwd", groups=4, per=6400, F=768, dtype="f16",
             post=True, gate=True, scale=True, carry=True),
        # float32, an odd width, a gate of every row's own
        dict(name="norm2bwd_1601x1000_rows_f32", op="norm2bwd", groups=1601, per=1, F=1000, dtype="f32",
             post=True, gate=True, scale=False, carry=False),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linearbwd", "ff", "ff", "ffbwd", "norm2", "norm2bwd"])
    dtype = rng.choice(["f16", "f16", "f32"])
    if op.startswith("norm2"):
        F = 8 * _log(rng, 1, 512)
        rows = _log(rng, 1, max(1, min(25600, 19000000 // F)))
        groups = rng.choice([1, min(rows, 4), rows])
        case = dict(op=op, groups=groups, per=rows // groups, F=F, dtype=dtype, post=rng.random() < 0.7,
                    gate=rng.random() < 0.7, scale=rng.random() < 0.6)
        if op == "norm2bwd":
            case["carry"] = rng.random() < 0.5
        return case
    K = 8 * _log(rng, 4, 256)
    N = 8 * _log(rng, 4, 512)
    # products of up to 25,600 rows; three and six of them in the gradients
    rows = _log(rng, 1, max(1, min(25600, 25600 * 768 * 2048 // (K * N))))
    if op == "linear":
        return dict(op=op, rows=rows, K=K, N=N, dtype=dtype, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "silu", "gelu", "logsigmoid"]), pre=rng.random() < 0.3,
                    residual=rng.random() < 0.5, alpha=rng.choice([1.0, 0.125, 1 / 16]))
    if op == "linearbwd":
        return dict(op=op, rows=rows, K=K, N=N, dtype=dtype, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "silu", "gelu", "logsigmoid"]),
                    alpha=rng.choice([1.0, 0.125, 1 / 16]))
    case = dict(op=op, rows=rows, K=K, F=N, dtype=dtype, act=rng.choice(["silu", "gelu"]))
    if op == "ff":
        case["parts"] = rng.random() < 0.5
    return case


def work(case):
    w = 2 if case["dtype"] == "f16" else 4
    op = case["op"]
    if op.startswith("norm2"):
        n = case["groups"] * case["per"] * case["F"]
        gates = case["groups"] * case["F"] if case["gate"] else 0
        if op == "norm2":
            return {"bytes": (4 * n + gates) * w, "flops": 10 * n}
        return {"bytes": ((5 + case["carry"]) * n + 2 * gates) * w, "flops": 25 * n}
    M, K = case["rows"], case["K"]
    N = case["F"] if op.startswith("ff") else case["N"]
    if op == "linear":
        return {"bytes": (M * K + N * K + M * N * (1 + case["residual"] + case["pre"])) * w,
                "flops": 2 * M * N * K}
    if op == "linearbwd":
        return {"bytes": (2 * M * K + 2 * N * K + M * N * (1 + (case["act"] != "none"))) * w,
                "flops": 4 * M * N * K}
    if op == "ff":
        return {"bytes": (M * K + 2 * N * K + M * N * (3 if case["parts"] else 1)) * w,
                "flops": 4 * M * N * K}
    return {"bytes": (2 * M * K + 4 * N * K + 3 * M * N) * w, "flops": 8 * M * N * K}


# --------------------------------------------------------------------------- inputs
def _type(case):
    return torch.float16 if case["dtype"] == "f16" else torch.float32


def _inputs(case, seed):
    """The case's inputs on the GPU, from the seed alone."""
    rng = torch.Generator(device="cuda").manual_seed(seed)
    t, op = _type(case), case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=rng, device="cuda")

    if op.startswith("norm2"):
        G, rows, F = case["groups"], case["groups"] * case["per"], case["F"]
        x = dict(x=(2 * normal(rows, F)).to(t), weight=1 + 0.1 * normal(F),
                 post=1 + 0.1 * normal(F) if case["post"] else None,
                 gate=(1 + 0.5 * normal(G, F)).to(t) if case["gate"] else None,
                 scale=0.1 + 0.02 * normal(F) if case["scale"] else None)
        stream = (4 * normal(rows, F)).to(t)
        if op == "norm2":
            x["residual"] = stream
        else:
            x["s"] = stream
            x["gy"] = normal(rows, F).to(t)
            x["gsum"] = normal(rows, F).to(t) if case["carry"] else None
        return x
    M, K = case["rows"], case["K"]
    x = dict(x=normal(M, K).to(t))
    if op.startswith("linear"):
        N = case["N"]
        x["weight"] = (normal(N, K) * K ** -0.5).to(t)
        x["bias"] = 0.1 * normal(N) if case["bias"] else None
        if op == "linear":
            x["residual"] = normal(M, N).to(t) if case["residual"] else None
        else:
            x["gy"] = normal(M, N).to(t)
            # what the forward kept
            x["pre"] = None if case["act"] == "none" else _affine(x).to(t)
        return x
    F = case["F"]
    x["gate_weight"], x["up_weight"] = ((normal(F, K) * K ** -0.5).to(t) for _ in range(2))
    if op == "ffbwd":
        x["a"], x["u"] = (_times(x["x"], x[n]).to(t) for n in ("gate_weight", "up_weight"))
        x["gh"] = normal(M, F).to(t)
    return x


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    return state


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


# --------------------------------------------------------------------------- the user's calls
def _own_act(gla, case):
    return {"none": gla.ACT_NONE, "silu": gla.ACT_SILU, "gelu": gla.ACT_GELU,
            "logsigmoid": gla.ACT_LOGSIGMOID}[case["act"]]


def _own_linear(x):
    from recurrent_vision_token_gla_amd import gla
    c = x["case"]
    return gla.linear(x["x"], x["weight"], x["bias"], act=_own_act(gla, c), alpha=c["alpha"],
                      residual=x["residual"], return_pre=c["pre"])


def _own_linearbwd(x):
    from recurrent_vision_token_gla_amd import gla
    c = x["case"]
    grads = gla.linear_bwd(x["x"], x["weight"], x["gy"], act=_own_act(gla, c), alpha=c["alpha"],
                           pre=x["pre"], need_bias=c["bias"])
    return grads if c["bias"] else grads[:2]


def _own_ff(x):
    from recurrent_vision_token_gla_amd import gla
    c = x["case"]
    return gla.gated_ff(x["x"], x["gate_weight"], x["up_weight"], act=_own_act(gla, c),
                        return_parts=c["parts"])


def _own_ffbwd(x):
    from recurrent_vision_token_gla_amd import gla
    return gla.gated_ff_bwd(x["x"], x["gate_weight"], x["up_weight"], x["a"], x["u"], x["gh"],
                            act=_own_act(gla, x["case"]))


def _own_norm2(x):
    from recurrent_vision_token_gla_amd import gla
    return gla.gated_add_rmsnorm(x["x"], x["residual"], x["weight"], EPS, post_weight=x["post"],
                                 gate=x["gate"], scale=x["scale"])


def _own_norm2bwd(x):
    from recurrent_vision_token_gla_amd import gla
    grads = gla.gated_add_rmsnorm_bwd(x["x"], x["s"], x["weight"], EPS, x["gy"], post_weight=x["post"],
                                      gate=x["gate"], scale=x["scale"], gsum=x["gsum"])
    return tuple(g for g in grads if g is not None)


# --------------------------------------------------------------------------- plain forms
def _times(x, w):
    return x.float() @ w.float().t()


def _affine(x):
    p = _times(x["x"], x["weight"])
    return p if x["bias"] is None else p + x["bias"]


def _act(p, kind):
    if kind == "silu":
        return p * torch.sigmoid(p)
    if kind == "gelu":
        return 0.5 * p * (1 + torch.erf(p * math.sqrt(0.5)))
    if kind == "logsigmoid":
        return p.clamp(max=0) - torch.log1p(torch.exp(-p.abs()))
    return p


def _slope(p, kind):
    if kind == "silu":
        sig = torch.sigmoid(p)
        return sig * (1 + p * (1 - sig))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(p * math.sqrt(0.5))) + p * torch.exp(-0.5 * p * p) / math.sqrt(2 * math.pi)
    return torch.sigmoid(-p)


def _plain_linear(x):
    c, t = x["case"], x["x"].dtype
    p = _affine(x)
    y = c["alpha"] * _act(p, c["act"])
    if x["residual"] is not None:
        y = y + x["residual"].float()
    return (y.to(t), p.to(t)) if c["pre"] else y.to(t)


def _plain_linearbwd(x):
    c, t = x["case"], x["x"].dtype
    g = c["alpha"] * x["gy"].float()
    if x["pre"] is not None:
        g = g * _slope(x["pre"].float(), c["act"])
    grads = ((g @ x["weight"].float()).to(t), (g.t() @ x["x"].float()).to(t))
    return grads + (g.sum(0),) if c["bias"] else grads


def _plain_ff(x):
    t = x["x"].dtype
    a, u = _times(x["x"], x["gate_weight"]), _times(x["x"], x["up_weight"])
    h = (_act(a, x["case"]["act"]) * u).to(t)
    return (h, a.to(t), u.to(t)) if x["case"]["parts"] else h


def _plain_ffbwd(x):
    a, u, gh, rows = (x[n].float() for n in ("a", "u", "gh", "x"))
    kind = x["case"]["act"]
    ga, gu = gh * u * _slope(a, kind), gh * _act(a, kind)
    gx = ga @ x["gate_weight"].float() + gu @ x["up_weight"].float()
    return tuple(g.to(x["x"].dtype) for g in (gx, ga.t() @ rows, gu.t() @ rows))


def _rstd(s):
    return 1 / (s.square().mean(-1, keepdim=True) + EPS).sqrt()


def _factor(x):
    """scale * gate of every row, [rows, F] or what broadcasts to it."""
    f = torch.ones((), device="cuda") if x["scale"] is None else x["scale"]
    if x["gate"] is not None:
        f = f * x["gate"].float().repeat_interleave(x["case"]["per"], 0)
    return f


def _plain_norm2(x):
    p = x["x"].float()
    if x["post"] is not None:
        p = p * _rstd(p) * x["post"]
    s = (x["residual"].float() + _factor(x) * p).to(x["x"].dtype)
    return (s.float() * _rstd(s.float()) * x["weight"]).to(s.dtype), s


def _norm_grad(s, g):
    """Gradient of s / rms(s) where g reaches it."""
    r = _rstd(s)
    n = s * r
    return r * (g - n * (g * n).mean(-1, keepdim=True))


def _plain_norm2bwd(x):
    t, s, m, gy = x["x"].dtype, x["s"].float(), x["x"].float(), x["gy"].float()
    gs = _norm_grad(s, gy * x["weight"])
    if x["gsum"] is not None:
        gs = gs + x["gsum"].float()
    n = m * _rstd(m) if x["post"] is not None else m
    p = n * x["post"] if x["post"] is not None else n
    gp = gs * _factor(x)
    gx = _norm_grad(m, gp * x["post"]) if x["post"] is not None else gp
    grads = [gx.to(t), gs.to(t), (gy * s * _rstd(s)).sum(0)]
    if x["post"] is not None:
        grads.append((gp * n).sum(0))
    if x["gate"] is not None:
        q = gs * p if x["scale"] is None else gs * p * x["scale"]
        grads.append(q.view(x["case"]["groups"], x["case"]["per"], -1).sum(1).to(t))
    if x["scale"] is not None:
        q = gs * p
        if x["gate"] is not None:
            q = q * x["gate"].float().repeat_interleave(x["case"]["per"], 0)
        grads.append(q.sum(0))
    return tuple(grads)


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, gradients from autograd."""
    x = {n: y.double() if torch.is_tensor(y) else y for n, y in _inputs(case, seed).items()}
    return globals()["_exact_" + case["op"]](case, x)


def _act64(p, kind):
    f = torch.nn.functional
    return {"none": lambda z: z, "silu": f.silu, "gelu": f.gelu, "logsigmoid": f.logsigmoid}[kind](p)


def _exact_linear(case, x):
    p = torch.nn.functional.linear(x["x"], x["weight"], x["bias"])
    y = _act64(p, case["act"]).mul(case["alpha"])
    y = y if x["residual"] is None else y.add(x["residual"])
    return (y, p) if case["pre"] else y


def _exact_linearbwd(case, x):
    if x["pre"] is None:
        gp = x["gy"] * case["alpha"]
    else:  # at the kept values of x W^T + bias
        pre = x["pre"].requires_grad_()
        gp, = torch.autograd.grad(_act64(pre, case["act"]), pre, x["gy"] * case["alpha"])
    rows, w = x["x"].requires_grad_(), x["weight"].requires_grad_()
    b = x["gy"].new_zeros(case["N"], requires_grad=True)
    grads = torch.autograd.grad(torch.nn.functional.linear(rows, w, b), (rows, w, b), gp)
    return grads if case["bias"] else grads[:2]


def _exact_ff(case, x):
    f = torch.nn.functional
    a, u = f.linear(x["x"], x["gate_weight"]), f.linear(x["x"], x["up_weight"])
    h = _act64(a, case["act"]).mul(u)
    return (h, a, u) if case["parts"] else h


def _exact_ffbwd(case, x):
    a, u = x["a"].requires_grad_(), x["u"].requires_grad_()
    ga, gu = torch.autograd.grad(_act64(a, case["act"]) * u, (a, u), x["gh"])
    rows, wg, wu = (x[n].requires_grad_() for n in ("x", "gate_weight", "up_weight"))
    f = torch.nn.functional
    return torch.autograd.grad((f.linear(rows, wg), f.linear(rows, wu)), (rows, wg, wu), (ga, gu))


def _rms64(s, w):
    return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * w


def _branch64(case, x):
    """[groups, per, F]: what the block adds to the stream."""
    p = x["x"] if x["post"] is None else _rms64(x["x"], x["post"])
    p = p.view(case["groups"], case["per"], case["F"])
    if x["gate"] is not None:
        p = p * x["gate"][:, None]
    return p if x["scale"] is None else p * x["scale"]


def _exact_norm2(case, x):
    s = x["residual"] + _branch64(case, x).reshape(x["residual"].shape)
    # the norm is of the sum as it is stored
    return _rms64(s.to(_type(case)).double(), x["weight"]), s


def _exact_norm2bwd(case, x):
    s, w = x["s"].requires_grad_(), x["weight"].requires_grad_()
    loss = (_rms64(s, w) * x["gy"]).sum()
    if x["gsum"] is not None:
        loss = loss + (s * x["gsum"]).sum()
    gs, gw = torch.autograd.grad(loss, (s, w))
    names = ["x"] + [n for n in ("post", "gate", "scale") if x[n] is not None]
    leaves = [x[n].requires_grad_() for n in names]
    gx, *rest = torch.autograd.grad(_branch64(case, x), leaves, gs.view(case["groups"], case["per"], -1))
    return (gx, gs, gw, *rest)
