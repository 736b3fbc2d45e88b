"""Who owns the workspace of a call: the binding's part, with plain host
memory in the device's place and the stream's state given."""
import contextlib
import weakref

import pytest
import torch

from w4a16_weight_only_dequant_amd import _lib


class Stream:
    cuda_stream = 0
    device_index = 0


@pytest.fixture
def streams(monkeypatch):
    """One stream, whose capture state the test sets."""
    state = {"stream": Stream(), "capturing": False}
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state["stream"])
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(_lib, "_workspaces", {})
    return state


@pytest.mark.parametrize("capturing", [True, False])
def test_a_captured_buffer_outlives_growth(streams, capturing):
    """A graph holds the address that a captured call was given: a larger call later must not free it."""
    ws = _lib.Workspace("cpu")
    streams["capturing"] = capturing
    held = weakref.ref(ws.get(2 << 20, streams["stream"]))
    streams["capturing"] = False
    assert held() is ws.get(1 << 20, streams["stream"])
    for size in (4 << 20, 8 << 20):
        larger = ws.get(size, streams["stream"])
        assert larger.numel() >= size and larger is not held()
    assert (held() is not None) == capturing


def test_a_buffer_grown_under_capture_outlives_growth(streams):
    ws = _lib.Workspace("cpu")
    eager = weakref.ref(ws.get(2 << 20, streams["stream"]))
    streams["capturing"] = True
    held = [weakref.ref(ws.get(size, streams["stream"])) for size in (3 << 20, 5 << 20)]
    streams["capturing"] = False
    ws.get(9 << 20, streams["stream"])
    assert eager() is None and all(h() is not None for h in held)


def test_default_under_capture_is_the_graphs_own(streams):
    """Neither an eager call nor another graph gets the memory of a captured call."""
    device = torch.device("cpu")
    eager = _lib._scratch(None, device, streams["stream"], 2 << 20)
    streams["capturing"] = True
    a = _lib._scratch(None, device, streams["stream"], 2 << 20)
    b = _lib._scratch(None, device, streams["stream"], 2 << 20)
    streams["capturing"] = False
    again = _lib._scratch(None, device, streams["stream"], 2 << 20)
    assert again is eager and len({t.data_ptr() for t in (eager, a, b)}) == 3
    own = _lib.Workspace("cpu")
    assert _lib._scratch(own, device, streams["stream"], 100) is own.buf
    assert _lib._scratch(own, device, streams["stream"], 0) is None
