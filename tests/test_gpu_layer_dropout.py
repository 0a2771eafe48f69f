"""Dropout against its definition: the same elements dropped, the others exact."""

import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


def want(x, p, seed, offset=0):
    f = ref.factors(x.numel(), p, seed, offset).view(x.shape)
    # float32 arithmetic, rounded once; a dropped element is +0 whatever x holds
    y = (x.float().cpu() * f.float()).to(x.dtype)
    return torch.where(f == 0, torch.zeros_like(y), y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2049, 5000])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_against_the_definition(lm, dtype, n, p):
    x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dtype).cuda()
    seed, offset = 0x123456789ABCDEF0, (1 << 32) - 3
    got = lm.dropout(x, p, seed, offset)
    assert got.dtype is dtype and torch.equal(got.cpu(), want(x, p, seed, offset))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_ends_and_what_is_not_finite(lm, dtype):
    x = torch.randn(999, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    assert torch.equal(lm.dropout(x, 0.0, 5), x)
    assert (lm.dropout(x, 1.0, 5) == 0).all() and not lm.dropout(x, 1.0, 5).signbit().any()
    assert torch.equal(lm.dropout(x, 1e-6, 5), x)  # t = 0
    x[3::7], x[5::7] = float("nan"), float("-inf")
    got, f = lm.dropout(x, 0.5, 5).cpu(), ref.factors(999, 0.5, 5)
    assert (got[f == 0] == 0).all() and torch.equal(got[f > 0].isnan(), x.cpu()[f > 0].isnan())
    for p in (0.25, 0.999, 1 - 2.0 ** -16):
        y = torch.ones(999, dtype=dtype, device="cuda")
        assert torch.equal(lm.dropout(y, p, -1, 3).cpu(), want(y, p, -1, 3))


def test_any_alignment_and_place(lm):
    flat = torch.randn(3000, generator=torch.Generator().manual_seed(2)).cuda()
    for base in (flat, flat.bfloat16()):
        for first in (0, 1, 2, 3, 5, 8):
            x = base[first:first + 1001]
            assert torch.equal(lm.dropout(x, 0.3, 11).cpu(), want(x, 0.3, 11))
            # the elements around an output stay as they were
            big = torch.full((1100,), 7.0, dtype=base.dtype, device="cuda")
            out = big[first:first + 1001]
            assert lm.dropout(x, 0.3, 11, out=out).data_ptr() == out.data_ptr() and torch.equal(out.cpu(), want(x, 0.3, 11))
            assert (big[:first] == 7).all() and (big[first + 1001:] == 7).all()
    mine = flat.clone()
    assert torch.equal(lm.dropout(mine, 0.3, 11, out=mine), lm.dropout(flat, 0.3, 11)) and lm.dropout(flat[:0], 0.3, 11).numel() == 0
    x = flat[:2400].view(2, 3, 400)
    assert torch.equal(lm.dropout(x, 0.3, 11).view(-1), lm.dropout(flat[:2400], 0.3, 11))
    # a second call that goes on where the first one ended
    assert torch.equal(lm.dropout(flat[800:1600], 0.3, 11, 100), lm.dropout(flat[:1600], 0.3, 11)[800:])


def test_the_gradient_is_the_same_call(lm):
    x = torch.randn(5000, generator=torch.Generator().manual_seed(3)).cuda()
    f = lm.dropout(torch.ones_like(x), 0.4, 77, 9)
    assert torch.equal(lm.dropout(x, 0.4, 77, 9), torch.where(f == 0, 0.0, x * f))


def test_the_share_that_is_dropped(lm):
    """n draws of probability t / 65536: within 6 standard deviations (a fixed seed: the same every time)."""
    n = 1 << 20
    for p in (0.01, 0.1, 0.5, 0.9):
        t = round(65536 * p) / 65536
        dropped = int((lm.dropout(torch.ones(n, device="cuda"), p, 4, 1 << 40) == 0).sum())
        assert abs(dropped - n * t) < 6 * (n * t * (1 - t)) ** 0.5, p


def test_state_on_the_device_and_graphs(lm):
    x = torch.randn(3001, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    state = torch.tensor([-12345, 70], dtype=torch.int64, device="cuda")
    assert torch.equal(lm.dropout(x, 0.2, state, 30), lm.dropout(x, 0.2, -12345, 100))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lm.dropout(x, 0.2, state, 30)
        state[1] += 376
    seen = []
    state.copy_(torch.tensor([-12345, 70]))
    for i in range(4):
        graph.replay()
        seen.append(out.clone())
        assert torch.equal(out, lm.dropout(x, 0.2, -12345, 100 + 376 * i))
        torch.cuda.synchronize()
    assert all(not torch.equal(a, b) for a, b in zip(seen, seen[1:]))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = lm.dropout(x, 0.2, 6)
    side.synchronize()
    assert torch.equal(got, lm.dropout(x, 0.2, 6))


def test_refusals(lm):
    x = torch.zeros(4, 6, device="cuda")
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    for fn, error in (
            (lambda: lm.dropout(x.half(), 0.1, 1), TypeError), (lambda: lm.dropout(x.t(), 0.1, 1), ValueError),
            (lambda: lm.dropout(x, -0.1, 1), ValueError), (lambda: lm.dropout(x, 1.1, 1), ValueError),
            (lambda: lm.dropout(x, float("nan"), 1), ValueError), (lambda: lm.dropout(x, 0.1, state.int()), TypeError),
            (lambda: lm.dropout(x, 0.1, state[:1]), ValueError), (lambda: lm.dropout(x, 0.1, state.cpu()), ValueError),
            (lambda: lm.dropout(x, 0.1, 1, out=x.bfloat16()), TypeError), (lambda: lm.dropout(x, 0.1, 1, out=x[:2]), ValueError),
            (lambda: lm.dropout(x.view(-1)[:20], 0.1, 1, out=x.view(-1)[4:]), ValueError),
            (lambda: lm.dropout(x.view(-1)[:4], 0.1, state, out=state.view(torch.float32)), ValueError)):
        with pytest.raises(error):
            fn()
    torch.cuda.synchronize()
