"""Cases of the framework's training and single-token operators, each in a plain
form (elementary torch operations) and as the calls a user makes.

op "bwd"       gradient of the key-only gated linear recurrence over a patch
               grid or a sequence (a grid of one row), from a carried state
op "step"      the recurrence for one new token per sequence, on a pool of
               states, optionally with the block's output gate
op "addnorm"   s = x + residual, y = RMSNorm(s) * w
op "addnorm8"  the same with y in 8 bits (e4m3) and a scale per row
op "normbwd"   gradient of addnorm
op "gatebwd"   gradient of the output gate RMSNorm(o) * w * silu(z)

`own` chooses between the two forms; prepare() makes the same inputs for both.
"""
import torch

own = False

EPS = 1e-6
L2R, R2L, T2B, B2T = 0, 1, 2, 3
C = 16  # tokens per chunk of the plain recurrence


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one 640x640 image (stride 16): the smallest training step, latency counts
        dict(name="bwd_40x40_h6", op="bwd", B=1, H=6, gh=40, gw=40, dk=64, dv=64, dtype="f16",
             gate="plain", dirs="1", carry=False),
        # one 1280x1280 image, column order
        dict(name="bwd_80x80_h6", op="bwd", B=1, H=6, gh=80, gw=80, dk=64, dv=64, dtype="f16",
             gate="plain", dirs="2", carry=False),
        # a block of the 12-block stack in training: four images, every direction,
        # channels that forget at once beside channels that keep
        dict(name="bwd_b4_80x80_h16", op="bwd", B=4, H=16, gh=80, gw=80, dk=64, dv=64, dtype="f16",
             gate="mixed", dirs="mix", carry=False),
        # a long ragged sequence in float32 at the pages' head shape, state carried in and out
        dict(name="bwd_seq4099_f32", op="bwd", B=2, H=4, gh=1, gw=4099, dk=32, dv=64, dtype="f32",
             gate="plain", dirs="0", carry=True),
        # one token of one stream
        dict(name="step_b1_h6", op="step", B=1, pad=0, slots=1, H=6, dk=64, dv=64, dtype="f16",
             gated=False),
        # serving: 250 streams of a pool of 512 and six padding rows, with the output gate
        dict(name="step_b256_h16_gated", op="step", B=256, pad=6, slots=512, H=16, dk=64, dv=64,
             dtype="f16", gated=True),
        # an odd batch in float32 at the pages' head shape
        dict(name="step_b37_h12_f32", op="step", B=37, pad=0, slots=64, H=12, dk=32, dv=64,
             dtype="f32", gated=False),
        # the norm before a mixer: one 1280x1280 image at the 768-wide block
        dict(name="addnorm_6400x768", op="addnorm", rows=6400, F=768, dtype="f16"),
        # the same for a batch of four, feeding 8-bit products
        dict(name="addnorm8_25600x768", op="addnorm8", rows=25600, F=768, dtype="f16"),
        # its gradient over the batch
        dict(name="normbwd_25600x768", op="normbwd", rows=25600, F=768, dtype="f16", carry=True),
        # float32 and an odd width
        dict(name="normbwd_1601x1000_f32", op="normbwd", rows=1601, F=1000, dtype="f32", carry=False),
        # the output gate's gradient on the stack's rows
        dict(name="gatebwd_b4_6400_h16", op="gatebwd", B=4, T=6400, H=16, dv=64, dtype="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["bwd", "bwd", "step", "addnorm", "addnorm8", "normbwd", "gatebwd"])
    dtype = rng.choice(["f16", "f16", "f32"])
    if op == "bwd":
        gh = rng.choice([1, _log(rng, 2, 128), _log(rng, 2, 128)])
        gw = _log(rng, 1, 16384) if gh == 1 else _log(rng, 2, 128)
        most = max(1, min(64, 200000 // (gh * gw)))
        B = _log(rng, 1, min(4, most))
        H = _log(rng, 1, max(1, most // B))
        return dict(op=op, B=B, H=H, gh=gh, gw=gw, dk=rng.choice([32, 64]), dv=rng.choice([32, 64]),
                    dtype=dtype, gate=rng.choice(["plain", "mixed"]),
                    dirs=rng.choice(["0", "1", "2", "3", "mix"]), carry=rng.random() < 0.5)
    if op == "step":
        B = _log(rng, 1, 256)
        pad = rng.choice([0, B // 5])
        return dict(op=op, B=B, pad=pad, slots=B - pad + rng.randrange(65), H=_log(rng, 1, 16),
                    dk=rng.choice([32, 64]), dv=rng.choice([32, 64]), dtype=dtype,
                    gated=rng.random() < 0.5)
    if op == "gatebwd":
        return dict(op=op, B=rng.choice([1, 2, 3]), T=_log(rng, 1, 6400), H=_log(rng, 1, 16),
                    dv=rng.choice([32, 64]), dtype=dtype)
    F = 8 * _log(rng, 1, 1024)
    rows = _log(rng, 1, max(1, min(25600, 20000000 // F)))
    case = dict(op=op, rows=rows, F=F, dtype=dtype)
    if op == "normbwd":
        case["carry"] = rng.random() < 0.5
    return case


def work(case):
    w = 2 if case["dtype"] == "f16" else 4
    op = case["op"]
    if op == "bwd":
        th = case["B"] * case["H"] * case["gh"] * case["gw"]
        dk, dv = case["dk"], case["dv"]
        states = 3 * case["B"] * case["H"] * dk * dv * 4 if case["carry"] else 0
        # q, k, gk, v, go in and four gradients out; two states read out of and three products
        # with the two states' updates, token by token
        return {"bytes": th * (6 * dk + 3 * dv) * w + states, "flops": th * 10 * dk * dv}
    if op == "step":
        bh = (case["B"] - case["pad"]) * case["H"]
        dk, dv = case["dk"], case["dv"]
        rows = 3 * dk + 2 * dv + (dv if case["gated"] else 0)
        return {"bytes": bh * (8 * dk * dv + rows * w), "flops": bh * 5 * dk * dv}
    if op == "gatebwd":
        n = case["B"] * case["T"] * case["H"] * case["dv"]
        return {"bytes": 5 * n * w, "flops": 20 * n}
    n = case["rows"] * case["F"]
    if op == "addnorm":
        return {"bytes": 4 * n * w, "flops": 5 * n}
    if op == "addnorm8":
        return {"bytes": 3 * n * w + n + 4 * case["rows"], "flops": 8 * n}
    return {"bytes": (4 if case["carry"] else 3) * n * w, "flops": 10 * n}


# --------------------------------------------------------------------------- inputs
def _type(case):
    return torch.float16 if case["dtype"] == "f16" else torch.float32


def _dirs(case):
    return [b % 4 for b in range(case["B"])] if case["dirs"] == "mix" else [int(case["dirs"])] * case["B"]


def _inputs(case, seed):
    """The case's inputs on the GPU, from the seed alone."""
    rng = torch.Generator(device="cuda").manual_seed(seed)
    t = _type(case)

    def normal(*shape):
        return torch.randn(shape, generator=rng, device="cuda")

    def log_decay(shape, gate):
        z = normal(*shape)
        if gate == "plain":
            return torch.nn.functional.logsigmoid(z) / 16
        strong = torch.rand((shape[0],) + (1,) * (len(shape) - 3) + tuple(shape[-2:]), generator=rng,
                            device="cuda") < 0.5
        return torch.where(strong, torch.nn.functional.logsigmoid(z - 4),
                           torch.nn.functional.logsigmoid(z + 4) / 16)

    if case["op"] == "bwd":
        B, H, T, dk, dv = case["B"], case["H"], case["gh"] * case["gw"], case["dk"], case["dv"]
        x = dict(q=normal(B, T, H, dk) * dk ** -0.5, k=normal(B, T, H, dk), v=normal(B, T, H, dv),
                 gk=log_decay((B, T, H, dk), case["gate"]), go=normal(B, T, H, dv))
        x = {n: y.to(t) for n, y in x.items()}
        x["s0"] = normal(B, H, dk, dv) if case["carry"] else None
        x["gs_final"] = normal(B, H, dk, dv) if case["carry"] else None
        return x
    if case["op"] == "step":
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        x = dict(q=normal(B, H, dk) * dk ** -0.5, k=normal(B, H, dk), v=normal(B, H, dv),
                 gk=log_decay((B, H, dk), "plain"))
        if case["gated"]:
            x["gate"] = normal(B, H, dv)
        x = {n: y.to(t) for n, y in x.items()}
        x["norm_weight"] = 1 + 0.1 * normal(dv)
        x["state"] = normal(case["slots"], H, dk, dv)
        order = torch.randperm(case["slots"], generator=rng, device="cuda")[:B - case["pad"]]
        x["slots"] = torch.cat([order, order.new_full((case["pad"],), -1)]).int()
        return x
    if case["op"] == "gatebwd":
        B, T, H, dv = case["B"], case["T"], case["H"], case["dv"]
        return dict(o=(2 * normal(B, T, H, dv)).to(t), gate=normal(B, T, H, dv).to(t),
                    norm_weight=1 + 0.1 * normal(dv), gy=normal(B, T, H, dv).to(t))
    rows, F = case["rows"], case["F"]
    x = dict(x=normal(rows, F).to(t), residual=(4 * normal(rows, F)).to(t), weight=1 + 0.1 * normal(F))
    if case["op"] == "normbwd":
        x = dict(s=x["residual"], weight=x["weight"], gy=normal(rows, F).to(t),
                 gs=normal(rows, F).to(t) if case["carry"] else None)
    return x


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if case["op"] == "step":  # rows of padding keep what they hold
        state["out"] = torch.zeros_like(state["v"])
    return state


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


# --------------------------------------------------------------------------- the user's calls
def _own_bwd(x):
    from recurrent_vision_token_gla_amd import gla
    c = x["case"]
    return gla.bwd(x["q"], x["k"], x["v"], x["gk"], x["go"], c["gh"], c["gw"], _dirs(c), s0=x["s0"],
                   gs_final=x["gs_final"], return_gs0=c["carry"])


def _own_step(x):
    from recurrent_vision_token_gla_amd import gla
    if x["case"]["gated"]:
        y = gla.step_gated(x["q"], x["k"], x["v"], x["gk"], x["gate"], x["norm_weight"], EPS,
                           x["state"], x["slots"], out=x["out"])
    else:
        y = gla.step(x["q"], x["k"], x["v"], x["gk"], x["state"], x["slots"], out=x["out"])
    return y, x["state"]


def _own_addnorm(x):
    from recurrent_vision_token_gla_amd import gla
    return gla.add_rmsnorm(x["x"], x["residual"], x["weight"], EPS)


def _own_addnorm8(x):
    from recurrent_vision_token_gla_amd import gla
    return gla.add_rmsnorm_q8(x["x"], x["residual"], x["weight"], EPS)


def _own_normbwd(x):
    from recurrent_vision_token_gla_amd import gla
    return gla.add_rmsnorm_bwd(x["s"], x["weight"], EPS, x["gy"], gsum=x["gs"])


def _own_gatebwd(x):
    from recurrent_vision_token_gla_amd import gla
    return gla.gate_bwd(x["o"], x["gate"], x["norm_weight"], EPS, x["gy"])


# --------------------------------------------------------------------------- plain forms
def _order(case):
    """[B, T] raster index of the token at each scan position."""
    gh, gw = case["gh"], case["gw"]
    raster = torch.arange(gh * gw, device="cuda")
    column = raster.view(gh, gw).t().reshape(-1)
    ways = torch.stack([raster, raster.flip(0), column, column.flip(0)])
    return ways[torch.tensor(_dirs(case), device="cuda")]


def _plain_bwd(x):
    """In chunks of C tokens: the pairs of a chunk through their decays, everything before and
    behind it through the states at its ends, which a triangular product over the chunks gives."""
    case, t = x["case"], x["q"].dtype
    B, T, H, dk = x["q"].shape
    N = -(-T // C)
    at = _order(case)[:, :, None, None]

    def chunks(a):  # [B, T, H, D] in raster order -> [B, H, N, C, D] in scan order, in 32 bits
        a = torch.take_along_dim(a.float(), at, 1).transpose(1, 2)
        return torch.nn.functional.pad(a, (0, 0, 0, N * C - T)).reshape(B, H, N, C, -1)

    def tokens(a):
        a = a.reshape(B, H, N * C, -1)[:, :, :T].transpose(1, 2)
        return torch.empty_like(a).scatter_(1, at.expand(a.shape), a).to(t).contiguous()

    q, k, v, go = (chunks(x[n]) for n in ("q", "k", "v", "go"))
    b = chunks(x["gk"]).double().cumsum(3)
    last = b[..., -1:, :]
    ends = last[..., 0, :].cumsum(2).transpose(2, 3)  # [B, H, dk, N] log-decay up to each chunk's end
    starts = ends - last[..., 0, :].transpose(2, 3)
    to_end, from_start = (last - b).exp().float(), b.exp().float()
    U = (k * to_end).transpose(3, 4) @ v
    R = (q * from_start).transpose(3, 4) @ go
    # between[n, m]: the decay from the end of chunk m to the start of chunk n > m
    between = starts[..., :, None] - ends[..., None, :]
    later = torch.ones(N, N, dtype=torch.bool, device="cuda").tril(-1)
    between = between.masked_fill(~later, -torch.inf).exp().float()
    S = (between @ U.transpose(2, 3)).transpose(2, 3)
    D = (between.transpose(3, 4).contiguous() @ R.transpose(2, 3)).transpose(2, 3)
    if case["carry"]:
        S = S + starts.exp().float().transpose(2, 3)[..., None] * x["s0"][:, :, None]
        D = D + (ends[..., -1:] - ends).exp().float().transpose(2, 3)[..., None] * x["gs_final"][:, :, None]
    pair = b[..., :, None, :] - b[..., None, :, :]
    causal = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    pair = pair.float().masked_fill(~causal[:, :, None], -torch.inf).exp()
    P = (go @ v.transpose(3, 4)).masked_fill(~causal, 0)
    A = (q[..., :, None, :] * k[..., None, :, :] * pair).sum(-1)
    pair = pair * P[..., None]
    gq = (pair * k[..., None, :, :]).sum(4) + from_start * (go @ S.transpose(3, 4))
    gkey = (pair * q[..., :, None, :]).sum(3) + to_end * (v @ D.transpose(3, 4))
    gv = A.transpose(3, 4) @ go + (k * to_end) @ D
    w = q * gq - k * gkey
    behind = ((last[..., 0, :].exp().float()[..., None] * S + U) * D).sum(-1)
    ggk = w.flip(3).cumsum(3).flip(3) + behind[..., None, :]
    outs = tuple(tokens(a) for a in (gq, gkey, gv, ggk))
    if case["carry"]:
        gs0 = (starts.exp().float().transpose(2, 3)[..., None] * R).sum(2)
        outs += (gs0 + ends[..., -1].exp().float()[..., None] * x["gs_final"],)
    return outs


def _norm(s):
    return s / (s.square().mean(-1, keepdim=True) + EPS).sqrt()


def _plain_step(x):
    rows = x["case"]["B"] - x["case"]["pad"]
    q, k, v, gk = (x[n][:rows].float() for n in ("q", "k", "v", "gk"))
    at = x["slots"][:rows].long()
    S = x["state"][at] * gk.exp()[..., None] + k[..., None] * v[..., None, :]
    o = (q[..., None] * S).sum(2)
    if x["case"]["gated"]:
        z = x["gate"][:rows].float()
        o = _norm(o) * x["norm_weight"] * z * torch.sigmoid(z)
    x["state"][at] = S
    x["out"][:rows] = o.to(x["out"].dtype)
    return x["out"], x["state"]


def _plain_addnorm(x):
    s = (x["x"].float() + x["residual"].float()).to(x["x"].dtype)
    return (_norm(s.float()) * x["weight"]).to(s.dtype), s


def _plain_addnorm8(x):
    s = (x["x"].float() + x["residual"].float()).to(x["x"].dtype)
    y = _norm(s.float()) * x["weight"]
    scale = y.abs().amax(-1) / 448
    return (y / scale[:, None]).to(torch.float8_e4m3fn), scale, s


def _plain_normbwd(x):
    s, gy = x["s"].float(), x["gy"].float()
    rstd = 1 / (s.square().mean(-1, keepdim=True) + EPS).sqrt()
    n, gn = s * rstd, gy * x["weight"]
    gx = rstd * (gn - n * (gn * n).mean(-1, keepdim=True))
    if x["gs"] is not None:
        gx = gx + x["gs"].float()
    return gx.to(x["s"].dtype), (gy * n).sum(0)


def _plain_gatebwd(x):
    o, z, gy, w = x["o"].float(), x["gate"].float(), x["gy"].float(), x["norm_weight"]
    rstd = 1 / (o.square().mean(-1, keepdim=True) + EPS).sqrt()
    n, sig = o * rstd, torch.sigmoid(z)
    gn = gy * w * z * sig
    go = rstd * (gn - n * (gn * n).mean(-1, keepdim=True))
    gz = gy * n * w * sig * (1 + z * (1 - sig))
    return go.to(x["o"].dtype), gz.to(x["o"].dtype), (gy * n * z * sig).sum((0, 1, 2))


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, token by token and with derivatives from autograd."""
    x = {n: y.double() if torch.is_tensor(y) and y.is_floating_point() else y
         for n, y in _inputs(case, seed).items()}
    return globals()["_exact_" + case["op"]](case, x)


def _exact_bwd(case, x):
    B, T, H, dk = x["q"].shape
    dv = case["dv"]
    if T > 17000:
        return None
    zero = x["q"].new_zeros(B, H, dk, dv)
    batch = torch.arange(B, device="cuda")
    rows = list(_order(case).t())
    S = x["s0"].clone() if case["carry"] else zero.clone()
    gq, gkey, gv, w = (torch.zeros_like(x[n]) for n in ("q", "k", "v", "gk"))
    for r in rows:
        S = S * x["gk"][batch, r].exp()[..., None] + x["k"][batch, r][..., None] * x["v"][batch, r][..., None, :]
        gq[batch, r] = (S @ x["go"][batch, r][..., None])[..., 0]
    E = x["gs_final"].clone() if case["carry"] else zero.clone()
    # dL/dgk_t = <S_T, dL/dS_T> + sum over t' >= t of q gq - k gk: in 64 bits nothing is lost
    total = (S * E).sum(-1)
    for r in reversed(rows):
        q, k = x["q"][batch, r], x["k"][batch, r]
        E = E + q[..., None] * x["go"][batch, r][..., None, :]
        gk_row = (E @ x["v"][batch, r][..., None])[..., 0]
        gkey[batch, r] = gk_row
        gv[batch, r] = (k[..., None, :] @ E)[..., 0, :]
        total = total + q * gq[batch, r] - k * gk_row
        w[batch, r] = total
        E = E * x["gk"][batch, r].exp()[..., None]
    return (gq, gkey, gv, w) + ((E,) if case["carry"] else ())


def _exact_step(case, x):
    state, out = x["state"].clone(), torch.zeros_like(x["v"])
    for row, slot in enumerate(x["slots"].tolist()):
        if slot < 0:
            continue
        state[slot] = torch.diag_embed(x["gk"][row].exp()) @ state[slot] + \
            x["k"][row][..., None] @ x["v"][row][..., None, :]
        o = (x["q"][row][..., None, :] @ state[slot])[..., 0, :]
        if case["gated"]:
            o = _gate64(o, x["gate"][row], x["norm_weight"])
        out[row] = o
    return out, state


def _gate64(o, z, w):
    return o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * w * torch.nn.functional.silu(z)


def _sum64(case, x):
    return (x["x"] + x["residual"]).to(_type(case)).double()


def _norm64(s, w):
    return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * w


def _exact_addnorm(case, x):
    s = _sum64(case, x)
    return _norm64(s, x["weight"]), s


def _exact_addnorm8(case, x):
    s = _sum64(case, x)
    y = _norm64(s, x["weight"])
    scale = y.abs().max(-1).values / 448
    return y / scale[:, None], scale, s


def _exact_normbwd(case, x):
    s, w = x["s"].requires_grad_(), x["weight"].requires_grad_()
    loss = (_norm64(s, w) * x["gy"]).sum()
    if x["gs"] is not None:
        loss = loss + (s * x["gs"]).sum()
    return torch.autograd.grad(loss, (s, w))


def _exact_gatebwd(case, x):
    o, z, w = x["o"].requires_grad_(), x["gate"].requires_grad_(), x["norm_weight"].requires_grad_()
    return torch.autograd.grad((_gate64(o, z, w) * x["gy"]).sum(), (o, z, w))
