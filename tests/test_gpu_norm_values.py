"""GPU: rows of the norm with NaN, infinities and squares at the ends of
float's range, as include/gla.h says."""
import numpy as np
import pytest
import torch

from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("F", [64, 1536])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_nan_and_infinity_stay_in_their_row(F, dtype):
    x = torch.ones(5, F, device="cuda", dtype=dtype)
    x[1, 3], x[2, 5], x[3, 7] = float("nan"), float("inf"), -float("inf")
    w = torch.ones(F, device="cuda")
    y, s = gla.add_rmsnorm(x, None, w, 1e-6)
    y8, sc, _ = gla.add_rmsnorm_q8(x, None, w, 1e-6)
    gx, gw = gla.add_rmsnorm_bwd(s, w, 1e-6, torch.ones_like(x))
    torch.cuda.synchronize()
    code = y8.float()
    assert torch.equal(s.isnan(), x.isnan())
    for out in (y, code):
        assert bool(out[1].isnan().all())
        for r, c in ((2, 5), (3, 7)):
            assert bool(out[r, c].isnan()) and int((out[r] != 0).sum()) == 1
        assert bool(out[[0, 4]].isfinite().all()) and torch.equal(out[0], out[4])
    assert sc[1:4].tolist() == [1, 1, 1] and bool((code[0] == 448).all())
    assert bool(gx[[0, 4]].isfinite().all()) and bool(gx[1].isnan().all())
    assert not bool(gw.isfinite().any())  # every column takes the row of NaN


@pytest.mark.parametrize("value", [2.0 ** -62, 1e-15, 1e15, 2.0 ** 58])
def test_float_rows_at_the_ends_of_the_range(value):
    """mean(s^2) from 2^-124 to 2^116, 1,000 of which still sum below 2^128: each
    of F/64 + 16 roundings is u, as for ordinary rows."""
    r = np.random.default_rng(3)
    x = (value * r.uniform(0.5, 1.0, (4, 1000))).astype(np.float32)
    want = x.astype(np.float64) / np.sqrt(np.mean(x.astype(np.float64) ** 2, 1, keepdims=True))
    y, _ = gla.add_rmsnorm(torch.from_numpy(x).cuda(), None, torch.ones(1000, device="cuda"), 0.0)
    torch.cuda.synchronize()
    assert float(np.max(np.abs(y.double().cpu().numpy() / want - 1))) <= (1000 / 64 + 17) * U
