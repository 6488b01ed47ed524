"""GPU: the products and their gradients on every kernel that the cost model picks
(test_product_plans.py), in whole numbers: sums below 2^24 are exact in float, by
any order and through the terms of float operands, so every output has one value,
rounded once."""
import pytest
import torch

from product_shapes import SHAPES
from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def whole(dtype, *shape, most=1):
    return torch.randint(-most, most + 1, shape, device="cuda", dtype=torch.int8).to(dtype)


def same(name, got, want):
    assert want.abs().max() < 1 << 24, name
    want = want.to(got.dtype)
    assert torch.equal(got, want), (name, (got != want).nonzero()[:4].tolist(), (got != want).sum().item())


def cases(call):
    return [(dtype, *s) for (c, dtype), shapes in SHAPES.items() if c == call for s in shapes]


@pytest.mark.parametrize("dtype,rows,K,N", cases("linear"))
def test_linear(dtype, rows, K, N):
    torch.manual_seed(rows + K + N)
    t = TYPES[dtype]
    x, w, res = whole(t, rows, K, most=3), whole(t, N, K), whole(t, rows, N, most=9)
    b = whole(torch.float32, N, most=20)
    plain = gla.linear(x, w)
    y, pre = gla.linear(x, w, b, alpha=0.5, residual=res, return_pre=True)
    torch.cuda.synchronize()
    want = x.double() @ w.double().t()
    same("plain", plain, want)
    same("pre", pre, want + b)
    same("y", y, 0.5 * (want + b) + res)


@pytest.mark.parametrize("dtype,rows,K,N", cases("gated"))
def test_gated(dtype, rows, K, N):
    torch.manual_seed(rows + K + N)
    t = TYPES[dtype]
    x, wg, wu = whole(t, rows, K), whole(t, N, K), whole(t, N, K)
    h, a, u = gla.gated_ff(x, wg, wu, act=gla.ACT_NONE, return_parts=True)
    torch.cuda.synchronize()
    wa, wu_ = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    same("a", a, wa)
    same("u", u, wu_)
    same("h", h, wa * wu_)


@pytest.mark.parametrize("dtype,rows,K,N", cases("linear_bwd"))
def test_linear_backward(dtype, rows, K, N):
    """With an activation, as the plans are for one: log sigmoid far to the left,
    where its slope is 1."""
    torch.manual_seed(rows + K + N)
    t = TYPES[dtype]
    x, w, gy = whole(t, rows, K), whole(t, N, K), whole(t, rows, N, most=3)
    pre = torch.full((rows, N), -1000.0, device="cuda", dtype=t)
    gx, gw, gb = gla.linear_bwd(x, w, gy, act=gla.ACT_LOGSIGMOID, alpha=0.5, pre=pre)
    torch.cuda.synchronize()
    g = gy.double()
    same("gx", gx, 0.5 * (g @ w.double()))
    same("gweight", gw, 0.5 * (g.t() @ x.double()))
    same("gbias", gb, 0.5 * g.sum(0))


@pytest.mark.parametrize("dtype,rows,K,N", cases("gated_bwd"))
def test_gated_backward(dtype, rows, K, N):
    torch.manual_seed(rows + K + N)
    t = TYPES[dtype]
    x, wg, wu, gh = whole(t, rows, K), whole(t, N, K), whole(t, N, K), whole(t, rows, N)
    a, u = whole(t, rows, N, most=3), whole(t, rows, N, most=3)
    gx, gwg, gwu = gla.gated_ff_bwd(x, wg, wu, a, u, gh, act=gla.ACT_NONE)
    torch.cuda.synchronize()
    ga, gu = gh.double() * u.double(), gh.double() * a.double()
    same("gx", gx, ga @ wg.double() + gu @ wu.double())
    same("ggate_weight", gwg, ga.t() @ x.double())
    same("gup_weight", gwu, gu.t() @ x.double())


@pytest.mark.parametrize("rows,K,N", [(1, 65536, 8), (1, 8, 65536), (5, 65536, 16), (16, 8, 65536), (17, 65536, 40),
                                      (40, 16, 65536), (300, 65536, 24), (300, 24, 65536)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_the_widest_rows(dtype, rows, K, N):
    test_linear(dtype, rows, K, N)
    test_gated(dtype, rows, min(K, 4096), N)
    test_linear_backward(dtype, rows, K, N)
    test_gated_backward(dtype, rows, K, N)
