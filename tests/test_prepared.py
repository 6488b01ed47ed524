"""The record of workspaces prepared for the single pass: no gradient takes a
workspace over any of their control words, wherever it starts.

CPU: the record itself, built with g++ on made-up addresses. GPU: the entry
points that ask it."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from recurrent_vision_token_gla_amd import gla
from recurrent_vision_token_gla_amd import workloads as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MIB = 1 << 20


def test_record_on_the_host(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "prepared")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-pthread",
                    "-I", os.path.join(ROOT, "recurrent_vision_token_gla_amd", "csrc"),
                    os.path.join(ROOT, "tests", "cpp", "prepared.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
def test_gradients_refuse_control_words_wherever_they_start():
    """Slices of a buffer around a prepared workspace: refused with E_ARG before
    any launch where they hold control words, and the forward is as it was."""
    B, gh, gw, H = 1, 8, 24, 2
    q, k, v, g = (torch.from_numpy(a).cuda() for a in W.make_inputs(B, gh * gw, H, 64, 64, np.float16, seed=41))
    go = torch.ones_like(v)
    rows = go.view(-1, 64)
    w = torch.ones(64, device="cuda")
    buf = torch.empty(12 * MIB, dtype=torch.uint8, device="cuda")
    ws = buf[4 * MIB:8 * MIB]
    gla.workspace_init(ws)
    want = gla.fwd(q, k, v, g, gh, gw, 0, workspace=ws, schedule=gla.SCHED_SINGLE_PASS)
    need = gla.bwd_workspace_bytes(B, H, gh, gw, 64, 64)
    small = gla.load().gla_add_rmsnorm_bwd_workspace_bytes(rows.shape[0], 64)
    calls = ((need, lambda x: gla.bwd(q, k, v, g, go, gh, gw, 0, workspace=x)),
             (small, lambda x: gla.add_rmsnorm_bwd(rows, w, 1e-6, rows, workspace=x)),
             (gla.load().gla_gate_bwd_workspace_bytes(rows.shape[0], 64),
              lambda x: gla.gate_bwd(rows, rows, w, 1e-6, rows, workspace=x)))
    assert need < 3 * MIB
    start = 4 * MIB
    for n, call in calls:
        n = (n + 255) // 256 * 256
        for at in (start, start + 256, start + gla.CTRL_BYTES - 256, start + 256 - n):
            with pytest.raises(gla.GLAError) as e:
                call(buf[at:at + n])
            assert e.value.status == gla.E_ARG, (n, at)
        for at in (start + gla.CTRL_BYTES, start - n):  # behind them, and up to them
            call(buf[at:at + n])
    torch.cuda.synchronize()
    assert not bool(ws[:gla.CTRL_BYTES].any())
    assert torch.equal(gla.fwd(q, k, v, g, gh, gw, 0, workspace=ws, schedule=gla.SCHED_SINGLE_PASS), want)
    gla.workspace_release(ws)
    calls[0][1](ws)


@pytest.mark.gpu
def test_a_freed_workspace_is_forgotten():
    """The record of a workspace ends with its memory, and not before: a view of
    it alone keeps it."""
    ws = torch.empty(MIB, dtype=torch.uint8, device="cuda")
    gla.workspace_init(ws)
    ptr, view = ws.data_ptr(), ws[256:]
    del ws
    assert gla.load().gla_workspace_is_prepared(ptr) == 1
    del view
    assert gla.load().gla_workspace_is_prepared(ptr) == 0
