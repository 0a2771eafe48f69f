"""The gated feed-forward block and its gradients against the definition in
float64, element by element within the bounds of their roundings."""

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


def make(n, width, hidden, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().cuda()  # noqa: E731
    return (t(n, width), t(hidden, width, std=2 * width ** -0.5), t(hidden, width, std=width ** -0.5),
            t(width, hidden, std=hidden ** -0.5), t(n, width))


def check(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all() and (over <= 0).all(), (what, float(over.max()), int((over > 0).sum()))


# sizes around the tiles (64, 128, 256) and steps of 64, the smallest, odd numbers of tokens
SIZES = [(1, 8, 8), (1, 64, 128), (3, 8, 72), (17, 264, 136), (64, 64, 64), (65, 72, 200), (127, 128, 128), (128, 136, 64),
         (129, 320, 264), (255, 64, 520), (257, 328, 256), (300, 1032, 72), (700, 200, 1000)]


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("n,width,hidden", SIZES)
def test_against_the_definition(lm, n, width, hidden, name):
    x, wg, wu, wd, dout = make(n, width, hidden)
    want, bound = ref.feed_forward(x, wg, wu, wd, name, dout)
    check(lm.feed_forward(x, wg, wu, wd, activation=name), want["out"], bound["out"], "out")
    out, kept = lm.feed_forward(x, wg, wu, wd, activation=name, keep=True)
    check(out, want["out"], bound["out"], "out, kept")
    check(kept, want["kept"], bound["kept"], "kept")
    got = lm.feed_forward_backward(dout, x, wg, wu, wd, kept, activation=name)
    for t, k in zip(got, ("dx", "dwg", "dwu", "dwd")):
        assert t.dtype is torch.bfloat16 and t.is_contiguous()
        check(t, want[k], bound[k], k)
