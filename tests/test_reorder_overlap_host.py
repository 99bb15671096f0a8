"""Host-side checks of what beam_reorder takes for overlapping tensors: views of
host memory, compared with the sets of bytes that they cover."""
import random

import pytest
import torch

from verify_dspark_markov_gb300 import binding


def covered(t):
    size = t.element_size()
    at = torch.zeros((), dtype=torch.int64)
    for n, s in zip(t.shape, t.stride()):
        at = at[..., None] + torch.arange(n) * s
    first = (t.data_ptr() + at.flatten() * size).tolist()
    return [a + i for a in first for i in range(size)]


def view(rng, base):
    """A slice of some of the dimensions, in some order."""
    for dim in range(base.dim()):
        n = base.shape[dim]
        kind = rng.random()
        if kind < 0.4:
            lo = rng.randrange(n)
            base = base.narrow(dim, lo, rng.randint(1, n - lo))
        elif kind < 0.5 and n > 1:
            base = base[(slice(None),) * dim + (slice(rng.randrange(2), None, 2),)]
    return base.permute(rng.sample(range(base.dim()), base.dim()))


def test_views_of_one_buffer():
    """Never taken for disjoint if they share a byte; and seldom refused for nothing."""
    rng, apart, refused = random.Random(1), 0, 0
    for _ in range(4000):
        base = torch.empty([rng.randint(1, 5) for _ in range(rng.randint(1, 4))], dtype=rng.choice([torch.uint8, torch.int32]))
        a, b = view(rng, base), view(rng, base)
        shared = bool(set(covered(a)) & set(covered(b)))
        said = binding._overlap(a, b)
        assert said == binding._overlap(b, a)
        assert said or not shared
        if not shared:
            apart += 1
            refused += said
        assert not binding._overlaps_itself(a)
    assert apart > 300 and refused < 0.1 * apart


def test_halves_of_a_double_buffer():
    buf = torch.empty((4, 2, 3, 5, 7))
    assert not binding._overlap(buf[:, 0], buf[:, 1])
    cache = torch.empty((2, 3, 4, 5, 32, 8))
    assert not binding._overlap(cache[..., :10, :], cache[..., 10:20, :])
    assert binding._overlap(cache[..., :10, :], cache[..., 9:20, :])
    assert binding._overlap(buf, buf[3, 1, 2, 4, 6])


def test_a_tensor_that_covers_a_byte_twice():
    x = torch.empty((3, 4))
    assert binding._overlaps_itself(x[:1].expand(3, 4)) and binding._overlaps_itself(x.as_strided((3, 4), (1, 1)))
    assert not binding._overlaps_itself(x.t()) and not binding._overlaps_itself(x[:, ::2])


@pytest.mark.parametrize("which", ["state", "another state", "another output", "itself", "parent"])
def test_what_is_refused(which, monkeypatch):
    """No kernel is reached: the outputs are looked at first."""
    monkeypatch.setattr(binding, "_dev", lambda t, name, dtype=None: t)
    monkeypatch.setattr(binding, "_Call", lambda stream, device: None)
    monkeypatch.setattr(binding, "load", lambda: pytest.fail("not refused"))
    a, b, room = torch.empty((2, 3, 4)), torch.empty((2, 3, 4)), torch.empty((2, 3, 4))
    parent, pair = torch.zeros((2, 3), dtype=torch.int32), torch.empty((2, 3, 4))
    states, out = {"state": ([a], [a]), "another state": ([a, b], [room, a]), "another output": ([a, b], [room, room]),
                   "itself": ([a], [pair[:, :1].expand(2, 3, 4)]),
                   "parent": ([torch.empty((2, 3), dtype=torch.int32)], [parent])}[which]
    with pytest.raises(ValueError, match="overlap"):
        binding.beam_reorder(states, parent, out=out)


def test_spans_of_a_descriptor():
    """The bytes that a state's descriptor spans are its tensor's."""
    rng = random.Random(2)
    for _ in range(300):
        outer, inner = rng.choice([(), (3,)]), rng.choice([(), (5,), (2, 6), (4, 3, 2)])
        B, W, M = rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 3)
        cut = (slice(None),) * (len(outer) + 2) + (slice(rng.randrange(2), None),) * min(1, len(inner))
        t = torch.empty((*outer, B, W, *inner), dtype=torch.int32)[cut]
        o = torch.empty((*outer, B, M, *inner), dtype=torch.int32)[cut]
        read, written, once = binding._spans(binding._state(t, o, len(outer), "t"), B, W, M)
        assert read == binding._extent(t) and written == binding._extent(o)
        assert once and not binding._overlaps_itself(o)
        if M > 1:
            twice = o.narrow(len(outer) + 1, 0, 1).expand(o.shape)
            assert not binding._spans(binding._state(t, twice, len(outer), "t"), B, W, M)[2]
