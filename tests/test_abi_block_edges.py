"""Edges of the products and norms between a block's mixers that show on the host
(CPU): no call here launches a kernel."""
import pytest

from recurrent_vision_token_gla_amd import gla
from test_abi_block import A, OK, _norm, _norm_bwd, lib  # noqa: F401


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_an_empty_batch_has_no_groups(lib, call):  # noqa: F811
    assert call(lib, rows=0, groups=0) == OK and call(lib, rows=0, groups=5) == OK
    assert call(lib, rows=4, groups=0) == A and call(lib, rows=0, groups=-1) == A
    assert gla.load().gla_gated_add_rmsnorm_bwd_workspace_bytes(0, 0, 64) == 0
