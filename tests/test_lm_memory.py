"""Which given outputs the binding of the language-model operators takes: the
test of shared memory against a list of every element's address (no GPU)."""

import itertools
import random

import pytest
import torch


@pytest.fixture(scope="module")
def lm():
    from newton_schulz_09_amd import lm as m
    return m


def addresses(t):
    """The byte addresses of a tensor's elements, with repetitions."""
    return [t.data_ptr() + t.element_size() * sum(i * s for i, s in zip(at, t.stride()))
            for at in itertools.product(*[range(n) for n in t.shape])]


def test_overlap_never_misses(lm):
    """Random views of one buffer: shared memory is always found."""
    rng = random.Random(0)
    flat = torch.zeros(4096, dtype=torch.bfloat16)
    found = said = 0
    for _ in range(3000):
        pair = []
        for _ in range(2):
            shape = [rng.choice([1, 2, 3]) for _ in range(4)]
            strides = [rng.choice([0, 1, 2, 4, 8, 12, 16, 32, 64, 96]) for _ in range(3)] + [1]
            pair.append(flat.as_strided(shape, strides, rng.randrange(0, 200)))
        a, b = pair
        shared = bool(set(addresses(a)) & set(addresses(b)))
        found += shared
        said += lm._overlap(a, b)
        assert lm._overlap(a, b) == lm._overlap(b, a) or shared
        assert not shared or lm._overlap(a, b), (a.shape, a.stride(), b.shape, b.stride())
        once = len(set(addresses(a))) == a.numel()
        assert once or lm._repeats(a), (a.shape, a.stride())
    assert 200 < found < said  # both answers occur


def test_views_that_programs_use_are_told_apart(lm):
    x = torch.zeros(2, 5, 8, 16, dtype=torch.bfloat16)
    parts = [x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]]            # q, k, v of one projection
    for a, b in itertools.permutations(parts, 2):
        assert not lm._overlap(a, b)
    assert lm._overlap(x[:, :, :5], x[:, :, 4:6])
    assert not lm._overlap(x[..., :8], x[..., 8:]) and lm._overlap(x[..., :9], x[..., 8:])
    assert not lm._overlap(x[:1], x[1:]) and not lm._overlap(x[:, :2], x[:, 2:])
    cache = torch.zeros(2, 3, 7, 2, 16)                         # keys and values, batch, positions, heads, size
    assert not lm._overlap(cache[0], cache[1]) and not lm._overlap(cache[0, :, :4], cache[0, :, 4:])
    assert not lm._overlap(torch.zeros(3), torch.zeros(3)) and not lm._overlap(x[:0], x)
    for t in (x, *parts, x.transpose(1, 2), x[:, ::2], x[:, :1].transpose(0, 3), cache[0]):
        assert not lm._repeats(t)
    for t in (x[:1].expand(2, 5, 8, 16), x[:, :, :1].expand_as(x), x.as_strided((2, 5, 8, 16), (640, 128, 8, 1))):
        assert lm._repeats(t)


def test_apart_allows_an_output_that_is_its_input(lm):
    x, y = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 4, 8)
    lm._apart(x, "out", (None, "a"), (y, "b"), (x, "c", True), (x.view(2, 3, 4, 8), "d", True))
    for other in ((x, "q"), (x[:, 1:], "q"), (x.transpose(0, 1).reshape_as(x).as_strided(x.shape, (12, 8, 24, 1)), "q")):
        if other[0].data_ptr() == x.data_ptr() or lm._overlap(x, other[0]):
            with pytest.raises(ValueError, match="out must not share memory with q"):
                lm._apart(x, "out", other)
    with pytest.raises(ValueError):
        lm._apart(x[:, :2], "out", (x[:, 1:], "q", True))
    with pytest.raises(ValueError):  # the same memory in another order
        lm._apart(x, "out", (x.as_strided(x.shape, (96, 32, 1, 4)), "q", True))
