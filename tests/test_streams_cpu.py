"""Memory that the bindings allocate for a call on another stream than the
current one: taken from that stream's pool, and known to be used on the current
one.  With stand-ins for torch's allocator and streams, so without a GPU."""
import contextlib
import types

import pytest
import torch

import dispatch_ffn_combine_gb300 as mk


@pytest.fixture
def log(monkeypatch):
    """What is allocated and recorded, and on which of the streams "current" and "other"."""
    events, now = [], ["current"]

    class Block:
        def record_stream(self, stream):
            events.append(("record", stream))

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(*shape, dtype=None, device=None):
        events.append(("empty", now[-1]))
        return Block()

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    return events


LIKE = types.SimpleNamespace(device="cuda:0")


def test_outputs_come_from_the_calls_stream(log):
    mk._new(None, torch.bfloat16, (4, 64), LIKE, "other")
    assert log == [("empty", "other"), ("record", "current")]
    del log[:]
    mk._new(None, torch.bfloat16, (4, 64), LIKE, None)
    assert log == [("empty", "current")]
    del log[:]
    t = object()
    assert mk._new(t, torch.bfloat16, (4, 64), LIKE, "other") is t and log == []


def test_workspaces_come_from_the_calls_stream(log):
    mk._workspace(None, 256, LIKE, "other")
    mk._workspace(None, 256, LIKE, None)
    assert log == [("empty", "other"), ("empty", "current")]
