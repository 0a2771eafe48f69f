"""The language-model operators on the GPU at the limits of their arguments:
caps and scales far from the usual ones, against float64 definitions."""

import pytest
import torch

from . import lm_bounds
from . import lm_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


def make(b, sq, sk, hq, hkv, d, seed=0, size=1.5):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().cuda()  # noqa: E731
    return t(b, sq, hq, d, std=size), t(b, sk, hkv, d), t(b, sk, hkv, d), t(b, sq, hq, d)


def check(lm, q, k, v, dout, softcap=0.0, slopes=None, scale=None, **mask):
    print(f"attention q {tuple(q.shape)} k {tuple(k.shape)} cap {softcap} scale {scale} {sorted(mask)}", flush=True)
    vis, pos = ref.visible(q.shape[0], q.shape[1], k.shape[1], **{n: t.cpu() if torch.is_tensor(t) else t for n, t in mask.items()})
    want, tol = lm_bounds.attention(q, k, v, dout, vis, pos, scale=scale, softcap=softcap, slopes=slopes)
    out, lse = lm.attention(q, k, v, softcap=softcap, slopes=slopes, scale=scale, **mask)
    grads = lm.attention_backward(dout, q, k, v, out, lse, softcap=softcap, slopes=slopes, scale=scale, **mask)
    torch.cuda.synchronize()
    for t, name in zip((out, lse, *grads), ("out", "lse", "dq", "dk", "dv")):
        ref.close(t, want[name], tol[name], name)


CAPS = [65.0, 100.0, 1e3, 1e4, 1e5, 1e6, 1e20, 2.0 ** 127 * 1.9]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("d", [64, 80, 128])
def test_large_caps(lm, cap, d):
    """A cap far above the scores changes nothing, and costs no accuracy either."""
    check(lm, *make(2, 150, 150, 4, 2, d), softcap=cap)


@pytest.mark.parametrize("cap", [80.0, 300.0, 1e4])
def test_large_caps_of_large_scores(lm, cap):
    """Scores on both sides of the cap."""
    check(lm, *make(1, 130, 130, 2, 1, 64, size=cap / 2), softcap=cap)


@pytest.mark.parametrize("cap", [100.0, 1e6])
def test_large_caps_with_masks(lm, cap):
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0]).cuda()
    check(lm, *make(2, 150, 150, 4, 2, 128), softcap=cap, slopes=slopes, window=70, causal=False)
    check(lm, *make(2, 3, 900, 4, 2, 64), softcap=cap, slopes=slopes)
    check(lm, *make(2, 1, 3000, 4, 1, 128), softcap=cap)


@pytest.mark.parametrize("cap", [1e-3, 1e-30, 1e-38, 1e-42])
def test_small_caps(lm, cap):
    """Scores of zero stay zero, however small the cap."""
    q, k, v, dout = make(1, 100, 100, 2, 1, 64)
    q[:, ::7] = 0
    check(lm, q, k, v, dout, softcap=cap)


@pytest.mark.parametrize("scale,size", [(2e-38, 2e18), (1e-37, 1e18), (3e-33, 1e16), (2.0 ** -101, 1e15), (2.0 ** -99, 1e15),
                                        (1e-6, 1e3), (1e6, 1e-3)])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(lm, scale, size, d):
    """Scores of ordinary size from a scale and heads that are not."""
    q, k, v, dout = make(1, 140, 140, 2, 1, d, size=1.0)
    check(lm, q * size, k * size, v, dout, scale=scale)
    check(lm, q * size, k * size, v, dout, scale=scale, window=30, causal=False)


def test_more_workgroups_than_one_grid_dimension_takes(lm):
    """2^24 workgroups of 256 threads: one key, so out = v, dv = dout, dq = dk = 0."""
    b, d = 2 ** 24 + 3, 8
    q, k, v, dout = (torch.randn(b, 1, 1, d, device="cuda").bfloat16() for _ in range(4))
    print(f"attention of {b} sequences of one token", flush=True)
    documents = torch.arange(b, dtype=torch.int32, device="cuda")[:, None]
    out, lse = lm.attention(q, k, v, documents=documents)
    assert torch.equal(out, v)
    # the score itself: 8 products and the factor in float32, and the logarithm back
    z = (q.double() * k.double()).sum(-1) / d ** 0.5
    room = 32 * 2.0 ** -24 * ((q.double() * k.double()).abs().sum(-1) + 1)
    assert bool(((lse.double().view(b, 1, 1) - z).abs() <= room).all())
    dq, dk, dv = lm.attention_backward(dout, q, k, v, out, lse, documents=documents)
    # P is 1 but for the exponent's rounding, 2^-20 at most; dP - delta the same of sum |dout v|
    mag = 2.0 ** -18 * (dout.double() * v.double()).abs().sum(-1, keepdim=True)
    assert bool(((dv - dout).abs().double() <= 2.0 ** -7 * dout.abs().double()).all())
    assert bool((dq.abs().double() <= mag * k.double().abs()).all()) and bool((dk.abs().double() <= mag * q.double().abs()).all())


def test_more_queries_than_one_grid_dimension_takes(lm):
    """33 queries a sequence, so whole blocks and not the split over keys."""
    b, s, d = 2 ** 24 + 1, 33, 8
    print(f"attention of {b} sequences of {s} tokens", flush=True)
    v = torch.randn(b, 1, 1, d, device="cuda").bfloat16()
    q = torch.randn(1, 1, 1, d, device="cuda").bfloat16().expand(b, s, 1, d)
    out, lse = lm.attention(q, v, v, causal=False)
    assert torch.equal(out, v.expand(b, s, 1, d))
    assert bool(torch.isfinite(lse).all())


def test_more_rows_than_one_grid_dimension_takes(lm):
    n, width = 2 ** 26 + 5, 65
    print(f"embedding of {n} tokens", flush=True)
    table = torch.randn(300, width, device="cuda").bfloat16()
    tokens = torch.randint(0, 300, (n,), dtype=torch.int32, device="cuda")
    out = lm.embedding(tokens, table)
    for at in range(0, n, 2 ** 23):
        assert torch.equal(out[at:at + 2 ** 23], table[tokens[at:at + 2 ** 23].long()]), at


@pytest.mark.parametrize("n,vocab", [(700, 2 ** 29 + 77), (3000, 2 ** 31 - 2)])
def test_larger_tables_than_one_grid_dimension_takes(lm, n, vocab):
    """Gradients of tables of one column: one launch, and sort, sums and zeros."""
    print(f"gradient of {n} tokens, {vocab} rows", flush=True)
    g = torch.Generator().manual_seed(1)
    rows = torch.tensor([0, 1, vocab // 2, vocab - 33, vocab - 2, vocab - 1])
    tokens = rows[torch.randint(0, 6, (n,), generator=g)]
    dout = torch.randint(-3, 4, (n, 1), generator=g).bfloat16()  # sums of whole numbers are exact
    grad = torch.full((vocab, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    lm.embedding_backward(dout.cuda(), tokens.cuda(), vocab, out=grad)
    want = torch.stack([dout[tokens == r].float().sum().bfloat16() for r in rows])
    assert torch.equal(grad[rows.cuda()][:, 0].cpu(), want)
    grad[rows.cuda()] = 0
    assert not any(bool(x.any()) for x in grad.split(2 ** 28))


@pytest.mark.parametrize("heads,d", [(25, 64), (3, 80), (5, 128)])
def test_odd_numbers_of_partial_results(lm, heads, d):
    """One token over 3200 keys in 3 chunks: an odd number of (row, chunk) pairs
    lies before the partial outputs."""
    check(lm, *make(1, 1, 3200, heads, heads, d))


@pytest.mark.parametrize("window", [2 ** 29, 2 ** 40, 2 ** 62])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_past_every_distance(lm, window, causal):
    """The same bits as without a window, also for positions far from the keys."""
    q, k, v, dout = make(3, 70, 200, 4, 2, 64)
    starts = torch.tensor([2 ** 31 - 1, -2 ** 31, 100], dtype=torch.int32).cuda()
    want = lm.attention(q, k, v, causal=causal, starts=starts)
    got = lm.attention(q, k, v, causal=causal, starts=starts, window=window)
    a = lm.attention_backward(dout, q, k, v, *want, causal=causal, starts=starts)
    b = lm.attention_backward(dout, q, k, v, *got, causal=causal, starts=starts, window=window)
    assert all(torch.equal(x, y) for x, y in zip((*want, *a), (*got, *b)))
