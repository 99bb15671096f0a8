"""GPU parity of dspark_distill_grad where its pipeline is in its steady state:
a dozen rows and more to a cluster, so that slices, barriers and the slots of the
exchange are used again and again, for each of the kernel's sizes and for
clusters of one, four and eight, with rows of weight 0 among the others.

The rows are repetitions of a few, which the plain 64-bit form computes; each
repetition is compared with the tolerances of test_distill_gpu.py (an element's
error is bounded by scale * weight / T times 1e-5 of the probabilities it is
formed from, bf16's rounding aside), whatever its place, alignment and
neighbours."""
import numpy as np
import pytest
import torch

import plain64
from test_distill_gpu import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_dspark_markov_gb300 as ds
    from verify_dspark_markov_gb300 import build
    build.build()
    ds.load()
    return ds


def unit_tolerance(b, grad):
    """Of a row's gradient at scale = weight = 1, apart from its rounding to the type."""
    p = np.zeros_like(grad)
    for i in range(len(grad)):
        ids = b.index[i].numpy()
        on = ids >= 0
        val = b.values[i].double().numpy()[on] / b.t
        p[i, ids[on]] = np.exp(val - float(b.lse[i]) if b.lse is not None else plain64.log_softmax(val))
    return 1e-5 * (np.abs(grad) + (2 * p + b.other_q()) / b.t)


def masks(kind, n, g):
    if kind == "none":
        return torch.zeros(n, dtype=torch.bool)
    if kind == "random":
        return torch.rand((n,), generator=g) < 0.5
    if kind == "few":  # one row in ten is read
        return torch.rand((n,), generator=g) < 0.9
    return torch.arange(n) // 100 % 2 == 0  # blocks


# (type, V, K, CTAs to a row, CTAs at once): the sizes the kernel is built for
SIZES = [(BF16, 2003, 20, 1, 304), (BF16, 4099, 256, 1, 304), (F32, 2048, 33, 1, 304),   # 4 vectors a thread
         (BF16, 8000, 64, 1, 304), (F32, 4095, 20, 1, 304),                             # 8
         (BF16, 16_001, 96, 1, 304), (F32, 8003, 20, 1, 304),                           # 16
         (BF16, 32_003, 64, 1, 152), (F32, 16_000, 256, 1, 152),                        # groups of 256 workers
         (BF16, 129_280, 64, 4, 152), (BF16, 129_283, 100, 4, 152), (F32, 65_001, 30, 4, 152),
         (BF16, 200_003, 20, 8, 152), (F32, 129_280, 100, 8, 152)]


@pytest.mark.parametrize("masked", ["none", "random", "few", "blocks"])
@pytest.mark.parametrize("dtype,v,k,ctas,at_once", SIZES)
def test_many_rows_to_a_cluster(ds, dtype, v, k, ctas, at_once, masked):
    base, n = 5, at_once // ctas * 13 + 3
    b = Batch(base, v, k, dtype, rest=v % 2 == 0, ragged=True, t=1.5 if k == 20 else 1.0)
    loss, grad, _, _ = plain64.distill(b.draft.double().numpy(), b.values.double().numpy(), b.index.numpy(),
                                       None if b.lse is None else b.lse.double().numpy(), None, b.t)
    tol = torch.from_numpy(unit_tolerance(b, grad)).to(DEV)
    grad = torch.from_numpy(grad).to(DEV)
    g = torch.Generator().manual_seed(v)
    pick = torch.randint(0, base, (n,), generator=g)
    weight = torch.rand((n,), generator=g) + 0.1
    off = masks(masked, n, g)
    weight[off] = 0.0
    args = [x[pick].to(DEV) for x in (b.draft, b.values, b.index)]
    got = ds.distill_grad(*args, lse=None if b.lse is None else b.lse[pick].to(DEV), weight=weight.to(DEV),
                          temperature=b.t, scale=b.scale)
    assert got["status"].eq(0).all()
    assert got["loss"][off].eq(0).all() and got["grad"][off].eq(0).all()
    for i in range(base):
        rows = torch.nonzero((pick == i) & ~off).flatten()
        np.testing.assert_allclose(got["loss"][rows.to(DEV)].double().cpu().numpy(), loss[i], rtol=1e-5, atol=1e-5)
        for part in rows.split(64):
            unit = (b.scale * weight[part].double()).to(DEV)[:, None]
            want = unit * grad[i]
            allowed = unit * tol[i] + 1e-35
            if dtype == BF16:
                allowed = allowed + want.abs() * 2.0 ** -8
            assert ((got["grad"][part.to(DEV)].double() - want).abs() <= allowed).all()
