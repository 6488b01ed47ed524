"""GPU: a gated call without its gate is refused, never taken for the ungated
one."""
import pytest
import torch

from recurrent_vision_token_gla_amd import gla

pytestmark = pytest.mark.gpu


def test_missing_gate_or_weight():
    q = torch.randn(2, 3, 32, device="cuda").half()
    state, w = torch.ones(2, 3, 32, 32, device="cuda"), torch.ones(32, device="cuda")
    out = torch.full_like(q, 7.0)
    for gate, weight in ((None, w), (q, None), (None, None)):
        with pytest.raises(ValueError):
            gla.step_gated(q, q, q, -q.abs(), gate, weight, 1e-6, state, out=out)
        with pytest.raises(ValueError):
            gla.gate_bwd(q, gate, weight, 1e-6, q)
    torch.cuda.synchronize()
    assert bool((state == 1).all()) and bool((out == 7).all())
    for call in (lambda: gla.add_rmsnorm(q, None, None, 1e-6), lambda: gla.add_rmsnorm_q8(q, None, None, 1e-6),
                 lambda: gla.add_rmsnorm_bwd(q, None, 1e-6, q), lambda: gla.add_rmsnorm_bwd(q, w, 1e-6, None)):
        with pytest.raises(ValueError):
            call()
