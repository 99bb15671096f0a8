"""GPU checks of dspark_beam_reorder on views that share a buffer without sharing
a byte: exact copies."""
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


def test_from_one_half_of_a_double_buffer_to_the_other(ds):
    """[layers, 2, B, W, heads, capacity, d]: back and forth."""
    g = torch.Generator(device=DEV).manual_seed(5)
    buf = torch.randint(0, 1000, (3, 2, 2, 4, 5, 16, 24), generator=g, device=DEV, dtype=torch.int32)
    parent = torch.tensor([[1, 1, 3, 0], [3, 2, 1, 0]], dtype=torch.int32, device=DEV)
    rows = torch.arange(2, device=DEV)[:, None]
    for step in range(4):
        src, dst = buf[:, step % 2], buf[:, 1 - step % 2]
        want, kept = src[:, rows, parent.long()], src.clone()
        ds.beam_reorder([src[..., :9, :]], parent, dim=1, out=[dst[..., :9, :]])
        assert torch.equal(dst[..., :9, :], want[..., :9, :]) and torch.equal(src, kept)
    with pytest.raises(ValueError):
        ds.beam_reorder([buf[:, 0]], parent, dim=1, out=[buf[:, 0]])
