"""Host-side check of beam_reorder on states without beams (no GPU: nothing is
enqueued)."""
import types

import pytest
import torch

from verify_dspark_markov_gb300 import binding


@pytest.fixture
def host(monkeypatch):
    call = types.SimpleNamespace(empty=lambda shape, dtype: torch.empty(shape, dtype=dtype), uses=lambda *t: None, ptr=0)
    monkeypatch.setattr(binding, "_dev", lambda t, name, dtype=None: t)
    monkeypatch.setattr(binding, "_Call", lambda stream, device: call)
    monkeypatch.setattr(binding, "load", lambda: None)


def test_no_beam_to_take_a_state_from(host):
    """The C entry point refuses W = 0; so does the call, which would have
    nothing to write into its outputs."""
    with pytest.raises(ValueError, match="beam"):
        binding.beam_reorder([torch.empty((2, 0, 4))], torch.full((2, 3), -1, dtype=torch.int32))


def test_nothing_to_write(host):
    (out,) = binding.beam_reorder([torch.empty((2, 0, 4))], torch.empty((2, 0), dtype=torch.int32))
    assert out.shape == (2, 0, 4)
    (out,) = binding.beam_reorder([torch.empty((0, 3, 4))], torch.empty((0, 5), dtype=torch.int32))
    assert out.shape == (0, 5, 4)
    (out,) = binding.beam_reorder([torch.empty((2, 3, 0))], torch.zeros((2, 5), dtype=torch.int32))
    assert out.shape == (2, 5, 0)
