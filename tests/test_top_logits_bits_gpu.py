"""GPU check that dspark_top_logits returns the logits as they are, bit for bit:
zeros of either sign, subnormal values, and the largest and lowest finite ones."""
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


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)])
@pytest.mark.parametrize("v", [7, 2003, 129_280])
def test_the_logits_as_they_are(ds, dtype, bits, v):
    g = torch.Generator().manual_seed(v)
    info = torch.finfo(dtype)
    some = torch.tensor([0.0, -0.0, info.smallest_normal / 4, -info.smallest_normal / 4, info.max, info.min], dtype=dtype)
    rows = [some[torch.randint(0, n, (v,), generator=g)] for n in (2, 4, 6)]
    rows.append(torch.where(torch.arange(v) % 3 == 0, torch.full((v,), -0.0), torch.randn(v, generator=g)).to(dtype))
    z = torch.stack(rows).to(DEV)
    for k in (1, 5, 200):
        got = ds.top_logits(z, k)
        kept = got["index"] >= 0
        want = torch.gather(z, 1, got["index"].clamp(min=0).long())
        assert torch.equal(got["values"].view(bits)[kept], want.view(bits)[kept])
        assert got["values"][~kept].eq(-torch.inf).all() and int(kept.sum()) == 4 * min(k, v)
