"""Graphs captured with the default workspace: each fills its own with zeros
whenever it is replayed, whichever is replayed first."""
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


def graphs(call, outs):
    """One graph to an output, captured one after the other."""
    every = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        every.append(g)
    return every


def replay_and_compare(every, outs, expected):
    for k in (1, 0, 1):  # the second first
        for t in outs[k].values():
            t.fill_(0)
        every[k].replay()
        torch.cuda.synchronize()
        for key, t in expected.items():
            assert torch.equal(outs[k][key], t), (k, key)


def test_distill_loss(ds):
    g = torch.Generator().manual_seed(0)
    z = torch.randn((40, 3001), generator=g).to(DEV)
    values, index = torch.topk(z, 8)
    index = index.to(torch.int32)
    draft = (z + torch.randn(z.shape, generator=g).to(DEV)).contiguous()
    expected = ds.distill_loss(draft, values, index)
    outs = [{k: torch.zeros_like(t) for k, t in expected.items()} for _ in range(2)]
    every = graphs(lambda out: ds.distill_loss(draft, values, index, out=out), outs)
    replay_and_compare(every, outs, expected)


def test_beam_select(ds):
    g = torch.Generator().manual_seed(1)
    z, score = torch.randn((6, 5, 2003), generator=g).to(DEV), torch.randn((6, 5), generator=g).to(DEV)
    expected = ds.beam_select(z, score, 10)
    outs = [{k: torch.zeros_like(t) for k, t in expected.items()} for _ in range(2)]
    every = graphs(lambda out: ds.beam_select(z, score, 10, out=out), outs)
    replay_and_compare(every, outs, expected)
