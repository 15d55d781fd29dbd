"""The binding's cached workspaces, without a GPU: what a captured graph has the
address of is not freed."""
from __future__ import annotations

import gc
import types
import weakref

import pytest
import torch

import linear_recurrence_scans_gb300 as mg

DEV = types.SimpleNamespace(index=0)


@pytest.fixture
def capture(monkeypatch):
    """Workspaces in host memory, and whether a capture is under way."""
    state = types.SimpleNamespace(on=False)
    stream = types.SimpleNamespace(synchronize=lambda: None, cuda_stream=7)
    monkeypatch.setattr(mg, "new_workspace", lambda n, device: torch.zeros(n, dtype=torch.uint8))
    monkeypatch.setattr(mg, "_ws_cache", {})
    monkeypatch.setattr(mg, "_ws_captured", {}, raising=False)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.on)
    return state


def test_a_captured_workspace_outlives_a_larger_call(capture):
    first = weakref.ref(mg._workspace(1000, DEV, 7, None))
    capture.on = True
    assert mg._workspace(500, DEV, 7, None) is first()
    capture.on = False
    larger = mg._workspace(1 << 20, DEV, 7, None)
    gc.collect()
    assert first() is not None and first() is not larger
    assert mg._workspace(1 << 19, DEV, 7, None) is larger


def test_a_workspace_that_no_graph_uses_is_freed(capture):
    first = weakref.ref(mg._workspace(1000, DEV, 7, None))
    mg._workspace(1 << 20, DEV, 7, None)
    gc.collect()
    assert first() is None


def test_no_workspace_grows_during_a_capture(capture):
    mg._workspace(1000, DEV, 7, None)
    capture.on = True
    with pytest.raises(RuntimeError, match="ws="):
        mg._workspace(1 << 20, DEV, 7, None)
    with pytest.raises(RuntimeError, match="ws="):
        mg._workspace(1000, DEV, 8, None)
