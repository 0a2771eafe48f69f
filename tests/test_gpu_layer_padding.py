"""Rows that only pad a batch: with zeros in what arrives for them (``dz`` and
``dx_out``, or ``dout``) and finite values, however large, in the tensors that the
gradients are computed from, they add nothing to the gradients that sum over
rows."""

import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


def check(got, want, bound, what):
    got = got.double().cpu()
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all() and (over <= 0).all(), (what, float(over.max()), int((over > 0).sum()))


@pytest.mark.parametrize("n", [40, 450, 5000])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_feed_forward(lm, n, name):
    """Gates up to 1e30 in padded tokens; every third token pads."""
    width, hidden = 72, 136
    g = torch.Generator().manual_seed(n)
    t = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(B)  # noqa: E731
    x, dout = t(n, width), t(n, width)
    wg, wu, wd = t(hidden, width, std=0.2), t(hidden, width, std=0.1), t(width, hidden, std=0.1)
    real = torch.arange(n) % 3 != 1
    want, bound = ref.feed_forward(x[real], wg, wu, wd, name, dout[real])
    dout[~real] = 0
    x, wg, wu, wd, dout = (v.cuda() for v in (x, wg, wu, wd, dout))
    out, kept = lm.feed_forward(x, wg, wu, wd, activation=name, keep=True)
    pad = (~real).cuda()
    x[pad] = 3e38
    kept[:, pad] = torch.where(torch.rand(3, int(pad.sum()), hidden, generator=g) < 0.5, -1e30, 1e30).to(B).cuda()
    dx, *dws = lm.feed_forward_backward(dout, x, wg, wu, wd, kept, activation=name)
    check(dx[real.cuda()], want["dx"], bound["dx"], "dx")
    assert (dx[pad] == 0).all()
    for got, k in zip(dws, ("dwg", "dwu", "dwd")):
        check(got, want[k], bound[k], k)


@pytest.mark.parametrize("gate", ["channel", "sequence", "full"])
@pytest.mark.parametrize("width", [96, 99, 1600])
@pytest.mark.parametrize("stream,block", [(B, B), (F, B), (F, F)])
@pytest.mark.parametrize("post", [False, True])
def test_norms(lm, stream, block, width, gate, post):
    """Streams and blocks of 1e30 (whose squares pass float32) and of zeros in the
    padded rows: the ends of the sequences."""
    b, s, lengths = 3, 21, (21, 5, 13)
    g = torch.Generator().manual_seed(width)
    t = lambda *sh, std=1.0, dtype=F: (torch.randn(*sh, generator=g) * std).to(dtype)  # noqa: E731
    x, xo, y = t(b, s, width, dtype=stream), t(b, s, width, dtype=stream), t(b, s, width, dtype=block)
    dz, dxo = t(b, s, width, dtype=block), t(b, s, width, dtype=stream)
    scale, prew, postw = 1 + t(width, std=0.2), 1 + t(width, std=0.2), 1 + t(width, std=0.2) if post else None
    gt = {"channel": lambda: t(width), "sequence": lambda: t(b, width), "full": lambda: t(b, s, width, dtype=block)}[gate]()
    pad = torch.arange(s)[None] >= torch.tensor(lengths)[:, None]
    for v in (dz, dxo):
        v[pad] = 0
    # the definition, in which a padded row is one of ordinary values
    want, bound = ref.residual_norm(x, y, gt, scale, postw, prew, post=post, xo=xo, dz=dz, dxo=dxo)
    for v in (x, xo, y):
        v[pad] = torch.where(torch.arange(int(pad.sum()))[:, None] % 3 == 0, 0.0, 1e30).to(v.dtype)
    c = lambda v: None if v is None else v.cuda()  # noqa: E731
    dx, dy, dgate, dscale, dpost, dpre = lm.residual_norm_backward(
        c(dz), c(dxo), c(xo), c(y), x=c(x), gate=c(gt), residual_scale=c(scale), post_weight=c(postw), pre_weight=c(prew),
        post=post)
    assert (dx[pad.cuda()] == 0).all() and (dy[pad.cuda()] == 0).all()
    for got, k, like in ((dx, "dx", x), (dy, "dy", y), (dgate, "dgate", gt), (dscale, "dscale", scale), (dpost, "dpostw", postw),
                         (dpre, "dprew", prew)):
        if like is not None:
            check(got, want[k], bound[k] + ref.rounding(like.dtype) * (want[k].abs() + bound[k]), k)
