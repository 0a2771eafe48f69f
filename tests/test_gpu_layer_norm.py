"""The norms around a block, with gate, residual scale and dropout, and their
gradients, against the definition in float64 within the bounds of float32."""

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
    assert got.shape == want.shape, what
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all() and (over <= 0).all(), (what, float(over.max()), int((over > 0).sum()))


def run(lm, b, s, width, stream=B, block=B, gate="none", scale=False, post=True, weights=True, p=0.0, has_y=True, eps=1e-6,
        seed=7):
    g = torch.Generator().manual_seed(seed)
    t = lambda *sh, std=1.0, dtype=F: (torch.randn(*sh, generator=g) * std).to(dtype).cuda()  # noqa: E731
    x, y = t(b, s, width, std=2.0, dtype=stream), t(b, s, width, std=0.5, dtype=block) if has_y else None
    prew = 1 + t(width, std=0.3) if weights else None
    postw = 1 + t(width, std=0.3) if weights and post and has_y else None
    sc = 1 + t(width, std=0.2) if scale else None
    gt = {"none": lambda: None, "channel": lambda: t(width), "sequence": lambda: t(b, width),
          "full": lambda: t(b, s, width, dtype=block)}[gate]()
    key, offset = 99 + seed, 5
    factor = ref.factors(x.numel(), p, key, offset).view(x.shape) if p else None
    kw = dict(gate=gt, residual_scale=sc, post_weight=postw, pre_weight=prew, post=post, eps=eps, p=p, seed=key,
              offset=offset)
    rkw = dict(gate=gt, scale=sc, postw=postw, prew=prew, post=post, eps=eps, factor=factor)
    xo, z = lm.residual_norm(x, y, dtype=None if has_y else block, **kw)
    assert xo.dtype is stream and z.dtype is block and xo.is_contiguous() and z.is_contiguous()
    want, bound = ref.residual_norm(x, y, **rkw)
    if not has_y:  # (the reference rounds z to the stream's type)
        bound["z"] = bound["z"] + ref.rounding(block) * want["z"].abs()
    check(xo, want["x_out"], bound["x_out"], "x_out")
    check(z, want["z"], bound["z"], "z")
    dz, dxo = t(b, s, width, dtype=block), t(b, s, width, dtype=stream)
    want, bound = ref.residual_norm(x if scale else None, y, xo=xo, dz=dz, dxo=dxo, **rkw)
    got = dict(zip(("dx", "dy", "dgate", "dscale", "dpostw", "dprew"),
                   lm.residual_norm_backward(dz, dxo, xo, y, x=x, **kw)))
    assert (got["dy"] is None) == (not has_y) and (got["dgate"] is None) == (gt is None)
    assert (got["dscale"] is None) == (sc is None) and (got["dpostw"] is None) == (postw is None)
    assert (got["dprew"] is None) == (prew is None)
    for k, like in (("dx", x), ("dy", y), ("dgate", gt), ("dscale", sc), ("dpostw", postw), ("dprew", prew)):
        if like is None:
            continue
        assert got[k].dtype is like.dtype
        last = ref.rounding(like.dtype) * (want[k].abs() + bound[k])
        check(got[k], want[k], bound[k] + last, k)


# widths around the pieces of a lane and the waves of a row, odd ones among them
@pytest.mark.parametrize("width", [1, 7, 8, 64, 100, 256, 257, 504, 512, 520, 768, 1024, 1032, 2047, 2048, 2056, 4096, 4104,
                                   8191, 8192])
@pytest.mark.parametrize("stream,block", [(B, B), (F, B), (F, F)])
def test_widths_and_types(lm, width, stream, block):
    run(lm, 2, 5, width, stream, block, gate="channel", scale=True, p=0.2)


@pytest.mark.parametrize("gate", ["none", "channel", "sequence", "full"])
@pytest.mark.parametrize("post,p", [(True, 0.0), (True, 0.3), (False, 0.0), (False, 0.3)])
@pytest.mark.parametrize("scale", [False, True])
@pytest.mark.parametrize("width", [96, 99])
def test_options(lm, gate, post, p, scale, width):
    run(lm, 3, 7, width, gate=gate, post=post, p=p, scale=scale)


@pytest.mark.parametrize("b,s", [(1, 1), (1, 2), (5, 1), (1, 700), (1100, 1), (600, 3), (1, 4999)])
@pytest.mark.parametrize("gate", ["channel", "sequence"])
def test_numbers_of_rows(lm, b, s, gate):
    run(lm, b, s, 72, F, F, gate=gate, scale=True)


# rows that share a wave: 8, 16 and 32 lanes each, and more rows than a turn of the workgroups takes
@pytest.mark.parametrize("width", [63, 64, 65, 120, 128, 129, 249, 256, 264])
@pytest.mark.parametrize("stream,block", [(B, B), (F, B)])
@pytest.mark.parametrize("b,s,gate", [(1, 1, "channel"), (3, 33, "sequence"), (2, 31, "full"), (5, 211, "sequence"), (1, 997, "channel")])
def test_narrow_rows(lm, b, s, gate, stream, block, width):
    run(lm, b, s, width, stream, block, gate=gate, scale=True, p=0.25)


@pytest.mark.parametrize("stream,block", [(B, B), (F, B), (F, F)])
@pytest.mark.parametrize("width", [96, 99, 2048])
def test_without_a_block(lm, stream, block, width):
    run(lm, 2, 9, width, stream, block, has_y=False)
    run(lm, 2, 9, width, stream, block, has_y=False, scale=True, weights=False)


def make(b, s, width, stream=B, block=B, seed=1):
    g = torch.Generator().manual_seed(seed)
    t = lambda *sh, dtype=F: torch.randn(*sh, generator=g).to(dtype).cuda()  # noqa: E731
    return t(b, s, width, dtype=stream), t(b, s, width, dtype=block), t(b, s, width, dtype=block), t(b, s, width, dtype=stream)


@pytest.mark.parametrize("stream,block", [(B, B), (F, B), (F, F)])
@pytest.mark.parametrize("width", [72, 75])
def test_layouts_and_outputs_in_place(lm, stream, block, width):
    """Rows inside wider tensors (at any alignment), outputs in place of what
    they replace, dimensions, and the memory around outputs."""
    x, y, dz, dxo = make(3, 7, width, stream, block)
    gate = (y * 0.5).contiguous()
    w = [torch.randn(width, generator=torch.Generator().manual_seed(i)).cuda() for i in range(3)]
    kw = dict(residual_scale=w[0], post_weight=w[1], pre_weight=w[2], p=0.25, seed=3)
    xo, z = lm.residual_norm(x, y, gate=gate, **kw)
    want = lm.residual_norm_backward(dz, dxo, xo, y, x=x, gate=gate, **kw)

    def inside(t, first, extra):
        big = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device=t.device)
        view = big[..., first:first + t.shape[-1]]
        view.copy_(t)
        return view

    for first, extra in ((0, 8), (8, 16), (3, 5), (1, 2)):
        xs, ys, gs, dzs, dxs, xos = (inside(t, first, extra) for t in (x, y, gate, dz, dxo, xo))
        got = lm.residual_norm(xs, ys, gate=gs, **kw)
        assert torch.equal(got[0], xo) and torch.equal(got[1], z)
        for a, c in zip(lm.residual_norm_backward(dzs, dxs, xos, ys, x=xs, gate=gs, **kw), want):
            assert torch.equal(a, c)
    mine, out = x.clone(), y.clone()
    got = lm.residual_norm(mine, out, gate=gate, x_out=mine, z_out=out, **kw)
    assert got[0] is mine and got[1] is out and torch.equal(mine, xo) and torch.equal(out, z)
    for give in ("dz", "y"):
        d1, d2, y2 = dxo.clone(), dz.clone(), y.clone()
        got = lm.residual_norm_backward(d2, d1, xo, y2, x=x, gate=gate, dx=d1, dy=d2 if give == "dz" else y2, **kw)
        assert got[0] is d1 and all(torch.equal(a, c) for a, c in zip(got, want))
    flat = lm.residual_norm(x.view(21, width), y.view(21, width), gate=gate.view(21, width), **kw)
    assert torch.equal(flat[0].view_as(x), xo)
    guard = torch.full((21 * width + 64,), 7.0, dtype=stream, device="cuda")
    lm.residual_norm(x, y, gate=gate, x_out=guard[:21 * width].view(x.shape), **kw)
    assert torch.equal(guard[:21 * width].view_as(x), xo) and (guard[21 * width:] == 7).all()
    # no gradient arrives at the stream: the same as zeros
    a = lm.residual_norm_backward(dz, None, xo, y, x=x, gate=gate, **kw)
    c = lm.residual_norm_backward(dz, torch.zeros_like(dxo), xo, y, x=x, gate=gate, **kw)
    assert all(torch.equal(i, j) for i, j in zip(a, c))


def test_other_rows_do_not_matter(lm):
    x, y, dz, dxo = make(1, 40, 96)
    kw = dict(gate=torch.ones(96, device="cuda"), p=0.25, seed=3)
    want = lm.residual_norm(x, y, **kw)
    grads = lm.residual_norm_backward(dz, dxo, want[0], y, **kw)[:2]
    bad = y.clone()
    bad[0, 5, 2], bad[0, 17, :] = float("nan"), float("inf")
    got = lm.residual_norm(x, bad, **kw)
    rows = [i for i in range(40) if i not in (5, 17)]
    assert all(torch.equal(a[:, rows], c[:, rows]) for a, c in zip(got, want)) and got[1][0, 5].isnan().all()
    more = lm.residual_norm_backward(dz, dxo, want[0], bad, **kw)[:2]
    assert all(torch.equal(a[:, rows], c[:, rows]) for a, c in zip(more, grads))
    # dropped elements are zero whatever the block's output holds (not normed: one element is no row's statistic)
    f = ref.factors(40 * 96, 0.25, 3).view(1, 40, 96).cuda()
    bad = torch.where(f == 0, torch.full_like(y, float("nan")), y)
    a = lm.residual_norm(x, bad, post=False, **kw)
    c = lm.residual_norm(x, torch.where(f == 0, torch.zeros_like(y), y), post=False, **kw)
    assert all(torch.equal(i, j) for i, j in zip(a, c))
    a = lm.residual_norm_backward(dz, dxo, c[0], bad, post=False, **kw)
    c = lm.residual_norm_backward(dz, dxo, c[0], torch.where(f == 0, torch.zeros_like(y), y), post=False, **kw)
    assert all(i is j is None or torch.equal(i, j) for i, j in zip(a, c))


@pytest.mark.parametrize("width", [64, 96, 99])
def test_rows_of_zeros_and_extreme_values(lm, width):
    x, y, dz, dxo = make(1, 6, width, F, F)
    y[0, 1] = 0
    x[0, 2], y[0, 2] = 0, 0
    got = lm.residual_norm(x, y, eps=1e-6)
    assert (got[1][0, 2] == 0).all() and all(torch.isfinite(t).all() for t in got)
    grads = lm.residual_norm_backward(dz, dxo, got[0], y, eps=1e-6)
    assert torch.isfinite(grads[0]).all() and torch.isfinite(grads[1]).all()
    # without eps a row of zeros is 0 / 0, and others are not touched
    a, c = lm.residual_norm(x, y, eps=0.0), lm.residual_norm(x[:, 3:].contiguous(), y[:, 3:].contiguous(), eps=0.0)
    assert a[1][0, 1:3].isnan().all() and torch.equal(a[1][:, 3:], c[1])
    run(lm, 2, 5, width, F, F, gate="channel", scale=True, eps=0.0)
    # far from 1, within what squares leave in float32
    for size in (1e-15, 1e15):
        a = lm.residual_norm(x * size, y, post=False, eps=0.0)[1][0, 0]
        v = (x * size + y)[0, 0].double()
        off = (a.double() - v / v.square().mean().sqrt()).abs().max()
        assert off < 1e-5, (size, float(off))


@pytest.mark.parametrize("gate", ["channel", "sequence"])
def test_empty(lm, gate):
    for b, s in ((0, 5), (3, 0)):
        x, y, dz, dxo = make(b, s, 64)
        w = torch.ones(64, device="cuda")
        kw = dict(gate=w if gate == "channel" else torch.ones(b, 64, device="cuda"), residual_scale=w, post_weight=w, pre_weight=w)
        xo, z = lm.residual_norm(x, y, **kw)
        assert xo.shape == z.shape == (b, s, 64)
        got = lm.residual_norm_backward(dz, dxo, xo, y, x=x, **kw)
        assert all((t == 0).all() for t in got) and got[2].shape == kw["gate"].shape


def test_same_bits_streams_and_graphs(lm):
    x, y, dz, dxo = make(4, 500, 136)
    gate = torch.randn(4, 136, generator=torch.Generator().manual_seed(2)).cuda()
    w = torch.ones(136, device="cuda")
    state = torch.tensor([5, 0], dtype=torch.int64, device="cuda")
    kw = dict(gate=gate, residual_scale=w, post_weight=w, pre_weight=w, p=0.1, seed=state)

    def step():
        xo, z = lm.residual_norm(x, y, **kw)
        return (xo, z, *lm.residual_norm_backward(dz, dxo, xo, y, x=x, **kw))

    want = [t.clone() for t in step()]
    assert all(torch.equal(a, c) for a, c in zip(step(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    here = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) and torch.equal(d, c) for a, d, c in zip(got, here, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        state[1] = 1000 * i
        y.copy_(make(4, 500, 136, seed=i)[1])
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(got, step())), i
        torch.cuda.synchronize()


def test_refusals(lm):
    x, y, dz, dxo = make(2, 5, 64)
    w = torch.ones(64, device="cuda")
    xo, z = lm.residual_norm(x, y)
    back = lambda **kw: lm.residual_norm_backward(dz, dxo, xo, y, **kw)  # noqa: E731
    for fn, error in (
            (lambda: lm.residual_norm(x.half(), y), TypeError), (lambda: lm.residual_norm(x, y.float()), TypeError),
            (lambda: lm.residual_norm(x, y[:, :4]), ValueError), (lambda: lm.residual_norm(x, y, dtype=F), TypeError),
            (lambda: lm.residual_norm(x, dtype=F), TypeError), (lambda: lm.residual_norm(x, gate=w), ValueError),
            (lambda: lm.residual_norm(x, p=0.1), ValueError), (lambda: lm.residual_norm(x, post_weight=w), ValueError),
            (lambda: lm.residual_norm(x, y, post=False, post_weight=w), ValueError),
            (lambda: lm.residual_norm(x, y, gate=w[:32]), ValueError), (lambda: lm.residual_norm(x, y, gate=w.bfloat16()), TypeError),
            (lambda: lm.residual_norm(x, y, gate=w.expand(3, 64).contiguous()), ValueError),
            (lambda: lm.residual_norm(x, y, gate=y.float()), TypeError), (lambda: lm.residual_norm(x, y, gate=3.0), TypeError),
            (lambda: lm.residual_norm(x, y, pre_weight=w.bfloat16()), TypeError),
            (lambda: lm.residual_norm(x, y, residual_scale=torch.ones(128, device="cuda")[::2]), ValueError),
            (lambda: lm.residual_norm(x.transpose(0, 1), y.transpose(0, 1)), ValueError),
            (lambda: lm.residual_norm(x, y, p=2.0), ValueError), (lambda: lm.residual_norm(x, y, eps=-1.0), lm.muon.MuonError),
            (lambda: lm.residual_norm(torch.zeros(2, 8200, device="cuda")), ValueError),
            (lambda: lm.residual_norm(x, y, x_out=y), ValueError), (lambda: lm.residual_norm(x, y, z_out=x), ValueError),
            (lambda: lm.residual_norm(x, y, x_out=z, z_out=z), ValueError),
            (lambda: lm.residual_norm(x, y, gate=y, z_out=y), ValueError),
            (lambda: back(residual_scale=w), TypeError), (lambda: back(dx=xo), ValueError), (lambda: back(dx=dz), ValueError),
            (lambda: back(dy=dxo), ValueError), (lambda: back(dx=dxo, dy=dxo), ValueError),
            (lambda: back(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), lm.muon.MuonError),
            (lambda: lm.residual_norm_backward(dz.float(), dxo, xo, y), TypeError),
            (lambda: lm.residual_norm_backward(dz, dxo[:, :3], xo, y), ValueError),
            (lambda: lm.residual_norm_backward(dz, dxo, xo, dy=y), ValueError)):
        with pytest.raises(error):
            fn()
    torch.cuda.synchronize()
