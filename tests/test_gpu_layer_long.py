"""The operators of a decoder layer on tensors whose offsets pass 32 bits: all
but the first and last rows are zeros, and those agree with a call of their own."""

import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu
B = torch.bfloat16


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    yield m
    torch.cuda.empty_cache()


def long(rows, width, few, dtype=B):
    """`few` (an even number of rows) at both ends of a long tensor of zeros."""
    x = torch.zeros(rows, width, dtype=dtype, device="cuda")
    h = len(few) // 2
    x[:h], x[-h:] = few[:h], few[h:]
    return x


def ends(x, few):
    h = len(few) // 2
    return torch.cat([x[:h], x[-h:]])


def rand(*shape, seed, std=1.0, dtype=B):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def test_dropout(lm):
    n, p, seed = (1 << 32) + 4099, 0.3, 77
    x = torch.ones(n, dtype=B, device="cuda")
    got = lm.dropout(x, p, seed)
    at = (1 << 32) - 4096  # the last elements, which begin with a block of the generator
    f = ref.factors(n - at, p, seed, at // 8)
    assert torch.equal(got[at:].cpu(), f.to(B)) and torch.equal(got[:4096].cpu(), ref.factors(4096, p, seed).to(B))


@pytest.mark.parametrize("gate", ["channel", "full"])
def test_norms(lm, gate):
    rows, width, p, seed = (1 << 20) + 13, 4104, 0.25, 5  # 4.3e9 elements
    few = [rand(6, width, seed=i) for i in range(5)]
    x, y, dz, dxo, gt = [long(rows, width, t) for t in few]
    vec = [1 + rand(width, seed=10 + i, std=0.3, dtype=torch.float32) for i in range(3)]
    kw = dict(post_weight=vec[0], pre_weight=vec[1], p=p, seed=seed)
    xo, z = lm.residual_norm(x, y, gate=gt if gate == "full" else vec[2], **kw)
    got = lm.residual_norm_backward(dz, dxo, xo, y, gate=gt if gate == "full" else vec[2], **kw)
    # the first and the last rows by themselves, the last with their own elements of the generator
    first = (rows - 3) * width // 8
    sums = None
    for part, offset in ((slice(0, 3), 0), (slice(3, 6), first)):
        a = [t[part].contiguous() for t in few]
        big = slice(0, 3) if offset == 0 else slice(rows - 3, rows)
        g = a[4] if gate == "full" else vec[2]
        xo1, z1 = lm.residual_norm(a[0], a[1], gate=g, offset=offset, **kw)
        assert torch.equal(xo[big], xo1) and torch.equal(z[big], z1)
        own = lm.residual_norm_backward(a[2], a[3], xo1, a[1], gate=g, offset=offset, **kw)
        for i in (0, 1, *((2,) if gate == "full" else ())):
            assert torch.equal(got[i][big], own[i]), i
        sums = own if sums is None else [None if s is None else s + t for s, t in zip(sums, own)]
    # of six rows a float32 sum of six: 6 half steps of the sum of magnitudes, which a column's cancellation
    # may leave far above its value, so the 2-norm over the columns counts
    for i in (4, 5, *((2,) if gate == "channel" else ())):
        assert (got[i].double() - sums[i].double()).norm() <= 6 * 2.0 ** -20 * sums[i].double().norm(), i


def test_feed_forward(lm):
    n, width, hidden = (1 << 21) + 777, 64, 1096  # 2.3e9 hidden values
    fx, fdout = rand(8, width, seed=1), rand(8, width, seed=2)
    wg, wu = rand(hidden, width, seed=3, std=0.25), rand(hidden, width, seed=4, std=0.125)
    wd = rand(width, hidden, seed=5, std=hidden ** -0.5)
    x, dout = long(n, width, fx), long(n, width, fdout)
    out, kept = lm.feed_forward(x, wg, wu, wd, keep=True)
    want, few = lm.feed_forward(fx, wg, wu, wd, keep=True)
    assert torch.equal(ends(kept.transpose(0, 1), fx), few.transpose(0, 1))  # one step of K: one order of sums
    assert torch.equal(lm.feed_forward(x, wg, wu, wd), out) and not out[4:-4].any()
    got = lm.feed_forward_backward(dout, x, wg, wu, wd, kept, dtype=torch.float32)
    own = lm.feed_forward_backward(fdout, fx, wg, wu, wd, few, dtype=torch.float32)
    assert not got[0][4:-4].any()
    for a, b, what in ((ends(out, fx), want, "out"), (ends(got[0], fx), own[0], "dx"), *zip(got[1:], own[1:], "guw")):
        # the same operands: sums in another order, and a rounding to bfloat16 that may fall the other way
        assert (a.double() - b.double()).norm() <= 2 * 2.0 ** -8 * b.double().norm(), what
