"""A workspace that grows: a captured graph replays into the buffer that it was
captured with, so that one is not given back while the workspace lives.  On the
host, with a fake of the capture's state."""
import gc
import weakref

import torch


def _buffers(monkeypatch, capturing):
    """Whether the first buffer lives on after the workspace has grown twice."""
    import quantized_gnn_message_gb300 as q
    state = {"capturing": False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    ws = q.Workspace("meta")
    first = ws.get(100)  # a call before: allocated outside the capture
    state["capturing"] = capturing
    assert ws.get(50) is first
    state["capturing"] = False
    alive = weakref.ref(first)
    del first
    assert ws.get(200).numel() >= 200 and ws.get(400).numel() >= 400 and ws.get(10).numel() >= 400
    gc.collect()
    there = alive() is not None
    del ws
    gc.collect()
    assert alive() is None
    return there


def test_a_captured_buffer_stays(monkeypatch):
    assert _buffers(monkeypatch, True)


def test_others_are_given_back(monkeypatch):
    assert not _buffers(monkeypatch, False)
