"""The feed-forward block at sizes that reach every tile and split of its
products (``layer_sizes.TILES``): each row and each column of every result against
float64, and the ragged ends, the first rows and some between element by element
within the bounds of their roundings."""

import pytest
import torch

from tests import layer_reference as ref
from tests.layer_sizes import TILES

pytestmark = pytest.mark.gpu
NAMES = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    yield m
    torch.cuda.empty_cache()


def make(n, width, hidden, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    return (t(n, width), t(hidden, width, std=2 * width ** -0.5), t(hidden, width, std=width ** -0.5),
            t(width, hidden, std=hidden ** -0.5), t(n, width))


def definition(x, wg, wu, wd, dout, name):
    x, wg, wu, wd, do = (t.double() for t in (x, wg, wu, wd, dout))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = ref.act(name, g)
    h, dh = a * u, do @ wd
    dg, du = dh * u * da, dh * a
    return {"out": h @ wd.t(), "kept": torch.stack([g, u, h]), "dx": dg @ wg + du @ wu, "dwg": dg.t() @ x, "dwu": du.t() @ x,
            "dwd": do.t() @ h}


def rows_and_columns(got, want, what):
    """Up to four roundings to bfloat16 lie between a result and its definition (gate
    or up, the hidden values or their gradient, twice for a sum of two products, the result), each
    at most 2^-8 of what is rounded; the matrices' random signs carry that to the
    2-norm of a row or column of 62 values and more.  A row, a column or a 16 x 16
    fragment of at most 6072 that is not there is off by 5% and more of the ones it lies in."""
    off = got.double() - want
    for dim in (-1, -2):
        far = off.norm(dim=dim) / want.norm(dim=dim)
        assert (far < 4 * 2.0 ** -8).all(), (what, dim, float(far.max()), int(far.argmax()))


def check(got, want, bound, what):
    got = got.double().cpu()
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all() and (over <= 0).all(), (what, float(over.max()), int((over > 0).sum()))


def some(n, seed):
    """The last values, which end in a ragged tile, the first, and some between."""
    at = torch.randint(n, (10,), generator=torch.Generator().manual_seed(seed)).tolist()
    return torch.tensor(sorted({*range(max(0, n - 18), n), 0, 1, *at})).cuda()


@pytest.mark.parametrize("which,n,width,hidden", [(i, *size) for i, size in enumerate(TILES)])
def test_every_tile(lm, which, n, width, hidden):
    name = NAMES[which % 4]
    x, wg, wu, wd, dout = make(n, width, hidden, which)
    out, kept = lm.feed_forward(x, wg, wu, wd, activation=name, keep=True)
    got = dict(zip(("dx", "dwg", "dwu", "dwd"), lm.feed_forward_backward(dout, x, wg, wu, wd, kept, activation=name)))
    got.update(out=out, kept=kept)
    want = definition(x, wg, wu, wd, dout, name)
    for k, t in got.items():
        rows_and_columns(t, want[k], k)
    del want
    single = lm.feed_forward_backward(dout, x, wg, wu, wd, kept, activation=name, dtype=torch.float32)[1:]
    # some tokens: their rows of out, kept and dx
    rows = some(n, which)
    want, bound = ref.feed_forward(x[rows], wg, wu, wd, name, dout[rows])
    for k in ("out", "dx"):
        check(got[k][rows], want[k], bound[k], k)
    check(kept[:, rows], want["kept"], bound["kept"], "kept")
    # some hidden values: their rows and columns of the matrices' gradients
    rows = some(hidden, which)
    cut = [t[rows].contiguous() for t in (wg, wu)] + [wd[:, rows].contiguous()]
    for dtype, grads in ((torch.bfloat16, [got[k] for k in ("dwg", "dwu", "dwd")]), (torch.float32, single)):
        want, bound = ref.feed_forward(x, *cut, name, dout, dtype=dtype)
        for k, t in zip(("dwg", "dwu", "dwd"), grads):
            assert t.dtype is dtype
            check(t[:, rows] if k == "dwd" else t[rows], want[k], bound[k], (k, dtype))
