"""Edges of the products and norms between a block's mixers that show on the host
(CPU): no call here launches a kernel."""
import os
import shutil
import subprocess

import pytest

from recurrent_vision_token_gla_amd import gla
from recurrent_vision_token_gla_amd.build import CSRC, HIPCC, ROOT
from test_abi_block import A, OK, _norm, _norm_bwd, lib  # noqa: F401


def host_program(name, tmp_path):
    """tests/cpp/<name>.hip compiled for the host alone, linked with the library."""
    if shutil.which(HIPCC) is None:
        pytest.skip("no hipcc")
    gla.load()
    obj, exe = str(tmp_path / (name + ".o")), str(tmp_path / name)
    subprocess.run([HIPCC, "-O1", "-std=c++17", "--offload-host-only", "-Wall", "-Werror", "-I", CSRC,
                    "-I", os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, "tests", "cpp", name + ".hip"),
                    "-o", obj], check=True)
    there = os.path.dirname(gla.LIB_PATH)
    subprocess.run([HIPCC, obj, "-L", there, "-l:" + os.path.basename(gla.LIB_PATH), "-Wl,-rpath," + there, "-o", exe],
                   check=True)
    return exe


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_an_empty_batch_has_no_groups(lib, call):  # noqa: F811
    assert call(lib, rows=0, groups=0) == OK and call(lib, rows=0, groups=5) == OK
    assert call(lib, rows=4, groups=0) == A and call(lib, rows=0, groups=-1) == A
    assert gla.load().gla_gated_add_rmsnorm_bwd_workspace_bytes(0, 0, 64) == 0


def test_launches_of_forward_products_are_in_range(tmp_path):
    """No launch has 2^32 threads, which HIP refuses, whatever fits the card."""
    exe = host_program("launches", tmp_path)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
