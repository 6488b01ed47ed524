"""Calls on a given stream leave the caller's device and stream as they were,
also where they fail."""
import contextlib
import types

import pytest
import torch

from recurrent_vision_token_gla_amd import gla


def test_contexts_are_left_where_entering_fails(monkeypatch):
    """CPU, with contexts that only count: whatever fails after the first one is
    open, none stays open."""
    opened = []

    @contextlib.contextmanager
    def context(name):
        if name == "refuses":
            raise RuntimeError(name)
        opened.append(name)
        try:
            yield
        finally:
            opened.remove(name)

    def refuse(stream):
        raise NotImplementedError

    monkeypatch.setattr(torch.cuda, "device", lambda device: context("device"))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    stream = types.SimpleNamespace(device="d", cuda_stream=7)
    bad = types.SimpleNamespace(is_cuda=True, device="d", record_stream=refuse)
    elsewhere = types.SimpleNamespace(is_cuda=False, device="cpu", record_stream=refuse)
    for name, inputs in (("stream", [bad]), ("refuses", [])):
        monkeypatch.setattr(torch.cuda, "stream", lambda s: context(name))
        with pytest.raises((NotImplementedError, RuntimeError)):
            with gla._There("d", stream, inputs):
                pass
        assert opened == []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: context("stream"))
    with gla._There("d", stream, [None, elsewhere]) as ptr:  # the call itself refuses a host tensor
        assert ptr == 7 and opened == ["device", "stream"]
    assert opened == []
    with pytest.raises(ValueError):
        with gla._There("other", stream, []):
            pass
    assert opened == []


@pytest.mark.gpu
def test_refused_calls_leave_the_current_stream():
    """A host tensor or a wrong one among the outputs, together with a stream:
    the binding's own ValueError, and the current stream as before."""
    s = torch.cuda.Stream()
    x = torch.randn(1, 20, 2, 32, device="cuda").half()
    rows, w = x.view(40, 32), torch.ones(32, device="cuda")
    pool = torch.zeros(1, 2, 32, 32, device="cuda")
    host = torch.empty_like(rows, device="cpu")
    row = x[:, 0].contiguous()
    g = -x.abs()
    calls = [lambda: gla.bwd(x, x, x, g, x, 4, 5, out=[torch.empty_like(x, device="cpu")] * 4, stream=s),
             lambda: gla.bwd(x, x, x, g, x, 4, 5, workspace=torch.empty(1 << 20, dtype=torch.uint8), stream=s),
             lambda: gla.bwd(x, x, x, g, x, 4, 5, return_gs0=True, gs0=torch.zeros(1, 2, 32, 32), stream=s),
             lambda: gla.step(row, row, row, -row.abs(), pool, out=torch.empty(1, 2, 32).half(), stream=s),
             lambda: gla.add_rmsnorm(rows, None, w, 1e-6, out=host, stream=s),
             lambda: gla.add_rmsnorm(rows, None, w, 1e-6, sum_out=host, stream=s),
             lambda: gla.add_rmsnorm_q8(rows, None, w, 1e-6, scales=torch.empty(40), stream=s),
             lambda: gla.add_rmsnorm_bwd(rows, w, 1e-6, rows, gweight=torch.empty(32), stream=s),
             lambda: gla.gate_bwd(rows, rows, w, 1e-6, rows, out=(host, host), stream=s)]
    before = torch.cuda.current_stream()
    assert before != s
    for call in calls:
        with pytest.raises(ValueError):
            call()
        assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
