"""GPU: the products and norms between a block's mixers at the edges of what they
take: empty batches."""
import pytest
import torch

from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gla.load()
    yield


def test_no_images_and_a_gate_of_each():
    """An empty batch has no row of a gate with one row for each image either."""
    w = torch.ones(64, device="cuda")
    for lead in ((0, 5), (0,)):
        x = torch.empty(*lead, 64, device="cuda").half()
        gate = torch.empty(0, 64, device="cuda").half()
        y, s = gla.gated_add_rmsnorm(x, x, w, EPS, gate=gate, scale=w)
        gx, gres, gw, gpost, ggate, gscale = gla.gated_add_rmsnorm_bwd(x, s, w, EPS, y, gate=gate, scale=w)
        torch.cuda.synchronize()
        assert y.shape == s.shape == gx.shape == gres.shape == x.shape and ggate.shape == gate.shape
        assert gpost is None and not gw.any() and not gscale.any()
    rows = torch.randn(3, 64, device="cuda").half()
    with pytest.raises(ValueError):  # rows without a gate of theirs
        gla.gated_add_rmsnorm(rows, rows, w, EPS, gate=rows[:0])
