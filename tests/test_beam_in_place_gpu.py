"""GPU check of dspark_beam_select writing the new scores over the old ones: the
same results as into a separate array, at every number of CTAs a beam, with beams
that offer no logits (finished, or of score -inf) beside others."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,W,V", [(1, 4, 129_280), (7, 5, 32_003), (20, 6, 5003), (60, 8, 515), (4, 64, 2003)])
def test_scores_in_place(ds, dtype, B, W, V):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = (3.0 * torch.randn((B, W, V), generator=g, device=DEV)).to(dtype)
    for step in range(40):
        score = torch.randn((B, W), generator=g, device=DEV) - 5.0
        off = torch.rand((B, W), generator=g, device=DEV)
        score[off < 0.4] = -torch.inf
        finished = ((off > 0.7) & (step % 2 == 0)).to(torch.uint8)
        want = ds.beam_select(z, score, W, finished=finished, eos=3)
        out = {k: torch.empty_like(t) for k, t in want.items()}
        out["scores"] = score
        ds.beam_select(z, score, W, finished=finished, eos=3, out=out)
        for key, t in want.items():
            assert torch.equal(out[key], t), key
