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
