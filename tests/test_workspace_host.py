"""Host-side checks of the workspaces of the row operators' calls (no GPU: the
buffers are on the host, and whether a stream is being captured is made up)."""
import pytest
import torch

from verify_dspark_markov_gb300 import binding


class Capture:
    on = False


@pytest.fixture
def capture(monkeypatch):
    state = Capture()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.on)
    monkeypatch.setattr(binding, "_default_ws", binding.Workspace())
    return state


def call():
    c = binding._Call.__new__(binding._Call)
    c.device, c.ptr, c.stream = torch.device("cpu"), 77, None
    return c


def test_a_captured_fill_is_not_taken_for_a_filled_buffer(capture):
    """The zero fill of a buffer made under capture runs with the graph, not
    now: another call, or another graph, must not find the buffer."""
    capture.on = True
    first, second = call().workspace(None, 5, 256), call().workspace(None, 5, 256)
    assert first.data_ptr() != second.data_ptr()
    capture.on = False
    eager = call().workspace(None, 5, 256)
    assert eager.data_ptr() not in (first.data_ptr(), second.data_ptr())
    assert call().workspace(None, 5, 256).data_ptr() == eager.data_ptr()


def test_a_graph_does_not_share_the_default_workspace_of_its_stream(capture):
    eager = call().workspace(None, 5, 256)
    capture.on = True
    assert call().workspace(None, 5, 256).data_ptr() != eager.data_ptr()


def test_an_explicit_workspace(capture):
    """One that was used before serves a capture; one that was not is not left
    with a buffer whose fill has yet to run."""
    ws = binding.Workspace()
    used = call().workspace(ws, 5, 256)
    capture.on = True
    assert call().workspace(ws, 5, 256).data_ptr() == used.data_ptr()
    larger = call().workspace(ws, 5, 512)
    assert larger.numel() == 512
    assert call().workspace(ws, 5, 512).data_ptr() != larger.data_ptr()
    capture.on = False
    assert call().workspace(ws, 5, 256).data_ptr() == used.data_ptr()
