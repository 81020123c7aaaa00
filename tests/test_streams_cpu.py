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


def test_layer_calls_allocate_on_their_stream(log):
    """The forward layer's helpers: outputs that a dict lacks, and the workspaces by size."""
    passed = object()
    res = mk._outputs({"row_token": passed}, {"row_token": (torch.int32, (4,)), "out": (torch.bfloat16, (4, 64))}, LIKE,
                      "other")
    assert res["row_token"] is passed and set(res) == {"row_token", "out"}
    mk._layer_workspace(None, 64, 128, 8, 2, 64, LIKE, "other")
    assert mk._layer_workspace(passed, 64, 128, 8, 2, 64, LIKE, "other") is passed
    assert log == [("empty", "other"), ("record", "current"), ("empty", "other")]


def test_no_binding_allocates_by_itself():
    """Every torch.empty of the module is one of the helpers': a call's memory has no other way past its stream."""
    import ast
    import inspect

    tree = ast.parse(inspect.getsource(mk))
    users = {f.name for f in ast.walk(tree) if isinstance(f, ast.FunctionDef)
             for c in ast.walk(f) if isinstance(c, ast.Attribute) and c.attr in ("empty", "empty_like", "zeros")
             and isinstance(c.value, ast.Name) and c.value.id == "torch"}
    assert users == {"_empty", "alloc_workspace", "alloc_dispatch_gemm_workspace"}
