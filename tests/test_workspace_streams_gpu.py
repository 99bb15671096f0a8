"""A workspace that a call on one stream made and a call on another still uses is
not handed out again by the allocator when it is dropped or outgrown."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_dspark_markov_gb300 as ds
    from verify_dspark_markov_gb300 import build
    build.build()
    ds.load()
    return ds


@pytest.mark.parametrize("first_on_side", [True, False])
def test_dropped_while_a_call_is_queued(ds, first_on_side):
    z, score = torch.randn((3, 4, 2003), device=DEV), torch.zeros((3, 4), device=DEV)
    want = ds.beam_select(z, score, 6)
    side, ws = torch.cuda.Stream(), ds.Workspace()
    torch.cuda.synchronize()
    here, there = (side, torch.cuda.current_stream()) if first_on_side else (torch.cuda.current_stream(), side)
    ds.beam_select(z, score, 6, workspace=ws, stream=here)
    torch.cuda.synchronize()
    (buf,) = ws._bufs.values()
    at, size = buf.data_ptr(), buf.numel()
    with torch.cuda.stream(there):
        torch.cuda._sleep(100_000_000)  # some tens of milliseconds
    got = ds.beam_select(z, score, 6, workspace=ws, stream=there)
    del ws, buf
    with torch.cuda.stream(here):
        other = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    for key, t in want.items():
        assert torch.equal(got[key], t), key
