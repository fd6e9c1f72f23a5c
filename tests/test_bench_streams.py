"""The benchmark's own streams start behind the stream that writes its
weights and tokens (no GPU: recording stand-ins)."""
import types

import pytest
import torch

import bench
from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I


class _Stream:
    def __init__(self, log):
        self.log = log

    def wait_stream(self, other):
        self.log.append(("wait", self, other))


@pytest.mark.parametrize("n_copy_streams", [1, 2])
def test_streams_wait_for_what_the_workload_was_made_by(monkeypatch, n_copy_streams):
    log = []
    current = _Stream(log)
    shape = I.LayerShape(T=4, H=64, I=64, E=4, k=2, S=0)
    tokens = torch.zeros((4, 64), dtype=torch.bfloat16)
    monkeypatch.setattr(torch.cuda, "Stream", lambda *a, **k: _Stream(log))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch.cuda, "Event", lambda *a, **k: types.SimpleNamespace(record=lambda *a: None))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(I, "make_layer", lambda *a, **k: log.append(("written",)) or types.SimpleNamespace(wr=None, bias=None))
    monkeypatch.setattr(I, "make_tokens", lambda *a, **k: log.append(("written",)) or tokens)
    monkeypatch.setattr(B, "Runtime", lambda *a, **k: types.SimpleNamespace(ctx=1, set_layer=lambda *a: None))
    monkeypatch.setattr(B, "RouteBuffers", lambda *a, **k: None)
    wl = bench.Workload(bench.Spec(shape, I.split_placement(4, 2, 1), 0.02, None), 1 << 20, n_copy_streams)
    last_write = max(i for i, e in enumerate(log) if e[0] == "written")
    behind = {id(e[1]) for e in log[last_write:] if e[0] == "wait" and e[2] is current}
    assert behind == {id(s) for s in [wl.compute] + wl.copies} and len(behind) == 1 + n_copy_streams
