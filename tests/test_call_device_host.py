"""The row operators' calls run on the current device alone: tensors or a stream
of another one are refused before anything is enqueued (no GPU: the devices are
made up)."""
import types

import pytest
import torch

from verify_dspark_markov_gb300 import binding


@pytest.fixture
def devices(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index)


def stream(index):
    return types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", index))


def test_the_current_device(devices):
    call = binding._Call(None, torch.device("cuda", 0))
    assert (call.stream, call.ptr) == (None, 100)
    side = stream(0)
    call = binding._Call(side, torch.device("cuda", 0))
    assert (call.stream, call.ptr) == (side, 5)


def test_another_device(devices):
    with pytest.raises(ValueError, match="current device"):
        binding._Call(None, torch.device("cuda", 1))
    with pytest.raises(ValueError, match="current device"):
        binding._Call(stream(1), torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        binding._Call(stream(1), torch.device("cuda", 0))
