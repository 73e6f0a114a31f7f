"""Workspace: which buffers it keeps."""

import weakref

import torch

import matrix_optimizers_sharded_amd as mo
from matrix_optimizers_sharded_amd import binding


def test_a_buffer_that_a_graph_writes_to_outlives_a_larger_call(monkeypatch):
    capturing = False
    monkeypatch.setattr(binding, "_capturing", lambda device: capturing, raising=False)
    ws = mo.Workspace(torch.device("cpu"))
    small = ws.get(1000)
    plain = weakref.ref(small)
    del small
    capturing = True
    first = ws.get(2000)
    capturing = False
    assert plain() is None                    # only eager calls had the smaller one
    at, held = first.data_ptr(), weakref.ref(first)
    del first
    assert ws.get(500).data_ptr() == at       # still the one in use
    second = ws.get(5000)                     # a larger eager call
    assert second.numel() == 5000 and second.data_ptr() != at
    assert held() is not None and held().data_ptr() == at
    dropped = weakref.ref(second)
    del second
    assert ws.get(9000).numel() == 9000
    assert dropped() is None                  # an eager call's buffer is let go
    assert held() is not None
