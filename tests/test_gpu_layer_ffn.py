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


def near(got, want, what):
    """Against a float32 result of the same bfloat16 operands: what bfloat16
    roundings on the way (at most 4: the hidden values, gate or up, their
    gradient, the result) do to the 2-norm, each at most 2^-8 relative."""
    off = (got.double() - want.double()).norm() / want.double().norm()
    assert off < 4 * 2.0 ** -8, (what, float(off))


def plain(x, wg, wu, wd, dout):
    """silu's block and gradients in float32 on the GPU, for sizes too large for float64 on the CPU."""
    x, wg, wu, wd, do = (t.float() for t in (x, wg, wu, wd, dout))
    g, u = x @ wg.t(), x @ wu.t()
    s = torch.sigmoid(g)
    h = g * s * u
    dh = do @ wd
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    return h @ wd.t(), dg @ wg + du @ wu, dg.t() @ x, du.t() @ x, do.t() @ h


# both tiles, products split over K (few tiles, long sums) and not, ragged ends of each
@pytest.mark.parametrize("n,width,hidden", [(70, 64, 8000), (5000, 64, 72), (9000, 264, 520), (2100, 1000, 3000), (4099, 768, 2048),
                                            (33, 2048, 5000), (3000, 3008, 64), (20000, 128, 136)])
def test_large_and_split_products(lm, n, width, hidden):
    x, wg, wu, wd, dout = make(n, width, hidden, 5)
    out, kept = lm.feed_forward(x, wg, wu, wd, keep=True)
    got = (out, *lm.feed_forward_backward(dout, x, wg, wu, wd, kept))
    for t, w, what in zip(got, plain(x, wg, wu, wd, dout), ("out", "dx", "dwg", "dwu", "dwd")):
        near(t, w, what)
    near(lm.feed_forward(x, wg, wu, wd), got[0].float(), "out, not kept")


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("width,hidden", [(8, 8), (40, 56), (72, 1000), (4096, 4104)])
def test_a_few_tokens(lm, n, width, hidden):
    """The path without kept values, up to 32 tokens and past it; of the largest
    matrices the few tokens that take it and those that take tiles."""
    x, wg, wu, wd, dout = make(n, width, hidden, 2)
    got = lm.feed_forward(x, wg, wu, wd)
    if width < 4096:
        want, bound = ref.feed_forward(x, wg, wu, wd, "silu")
        check(got, want["out"], bound["out"], "out")
    else:
        near(got, plain(x, wg, wu, wd, dout)[0], "out")
    if n <= 16 and width < 4096:  # the same kernels: the same bits for each token
        assert torch.equal(got[:1], lm.feed_forward(x[:1].contiguous(), wg, wu, wd))


def test_layouts(lm):
    """Halves of one matrix, rows inside wider ones, leading dimensions, outputs
    given, float32 gradients; NaN around what the arguments cover."""
    n, width, hidden = 130, 72, 200
    x, wg, wu, wd, dout = make(n, width, hidden)
    out, kept = lm.feed_forward(x, wg, wu, wd, keep=True)
    want = lm.feed_forward_backward(dout, x, wg, wu, wd, kept)

    def inside(t, extra):  # t's values in a wider matrix of NaN
        big = torch.full((t.shape[0] + 3, t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
        view = big[:t.shape[0], 8:8 + t.shape[1]] if extra > 8 else big[:t.shape[0], :t.shape[1]]
        view.copy_(t)
        return view

    both = torch.cat([wg, wu])
    xs, dos, wds = inside(x, 8), inside(dout, 24), inside(wd, 16)
    wide = inside(both, 32)
    for g, u in ((both[:hidden], both[hidden:]), (wide[:hidden], wide[hidden:])):
        o, k = lm.feed_forward(xs, g, u, wds, keep=True)
        assert torch.equal(o, out) and torch.equal(k, kept)
        for a, b in zip(lm.feed_forward_backward(dos, xs, g, u, wds, k), want):
            assert torch.equal(a, b)
    x3 = x.view(2, 5, 13, width)
    o, k = lm.feed_forward(x3, wg, wu, wd, keep=True)
    assert o.shape == x3.shape and torch.equal(o.view_as(out), out)
    got = lm.feed_forward_backward(dout.view_as(x3), x3, wg, wu, wd, k)
    assert got[0].shape == x3.shape and torch.equal(got[0].view_as(x), want[0]) and torch.equal(got[1], want[1])
    # the rows behind an output stay as they were
    for tokens in (n, 20):
        guard = torch.full((n + 40, width), 7.0, dtype=torch.bfloat16, device="cuda")
        assert lm.feed_forward(x[:tokens], wg, wu, wd, out=guard[:tokens]).data_ptr() == guard.data_ptr()
        assert torch.equal(guard[:tokens], lm.feed_forward(x[:tokens].contiguous(), wg, wu, wd)) and (guard[tokens:] == 7.0).all()
    f32 = lm.feed_forward_backward(dout, x, wg, wu, wd, kept, dtype=torch.float32)
    for a, b in zip(f32[1:], want[1:]):
        assert a.dtype is torch.float32 and torch.equal(a.bfloat16(), b)  # the same sums, not rounded


def test_other_rows_do_not_matter(lm):
    """Infinities and NaN in one token reach that token's result alone (and the
    matrices' gradients, as in any sum)."""
    for n, keep in ((300, True), (24, False)):
        x, wg, wu, wd, dout = make(n, 64, 136)
        want = lm.feed_forward(x, wg, wu, wd, keep=keep)
        bad = x.clone()
        bad[7, 3], bad[20, :] = float("nan"), float("inf")
        got = lm.feed_forward(bad, wg, wu, wd, keep=keep)
        rows = [i for i in range(n) if i not in (7, 20)]
        a, b = (got[0], want[0]) if keep else (got, want)
        assert torch.equal(a[rows], b[rows]) and a[7].isnan().all()


def test_no_tokens(lm):
    x, wg, wu, wd, dout = make(0, 64, 72)
    out, kept = lm.feed_forward(x, wg, wu, wd, keep=True)
    assert out.shape == (0, 64) and kept.shape == (3, 0, 72) and lm.feed_forward(x, wg, wu, wd).shape == (0, 64)
    for dtype in (torch.bfloat16, torch.float32):
        dx, *dws = lm.feed_forward_backward(dout, x, wg, wu, wd, kept, dtype=dtype)
        assert dx.shape == (0, 64) and all(t.dtype is dtype and t.shape == w.shape and (t == 0).all() for t, w in zip(dws, (wg, wu, wd)))


def test_same_bits_streams_and_graphs(lm):
    x, wg, wu, wd, dout = make(1500, 264, 520)

    def step():
        out, kept = lm.feed_forward(x, wg, wu, wd, activation="gelu", keep=True)
        return (out, *lm.feed_forward_backward(dout, x, wg, wu, wd, kept, activation="gelu"), lm.feed_forward(x[:9], wg, wu, wd))

    want = [t.clone() for t in step()]
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    here = step()  # the two run at once, each with a workspace of its own
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) and torch.equal(c, b) for a, c, b in zip(got, here, want))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.cuda.graph(other):
        more = step()
    fresh = make(1500, 264, 520, 9)
    for i in range(4):
        src = fresh if i & 1 else make(1500, 264, 520)
        for t, s in zip((x, wg, wu, wd, dout), src):
            t.copy_(s)
        graph.replay()
        other.replay()
        eager = step()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, c, b in zip(got, more, eager)), i
        torch.cuda.synchronize()


def test_refusals(lm):
    x, wg, wu, wd, dout = make(20, 64, 72)
    out, kept = lm.feed_forward(x, wg, wu, wd, keep=True)
    flat = torch.zeros(20 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    for fn, error in (
            (lambda: lm.feed_forward(x.float(), wg, wu, wd), TypeError),
            (lambda: lm.feed_forward(x, wg.float(), wu, wd), TypeError),
            (lambda: lm.feed_forward(x, wg, wu[:64], wd), ValueError),
            (lambda: lm.feed_forward(x, wg, wu, wd.t()), ValueError),
            (lambda: lm.feed_forward(x[:, :56], wg, wu, wd), ValueError),
            (lambda: lm.feed_forward(x, wg, torch.zeros(72, 72, dtype=torch.bfloat16, device="cuda")[:, :64], wd), ValueError),
            (lambda: lm.feed_forward(x, wg, wu, wd, activation="tanh"), ValueError),
            (lambda: lm.feed_forward(x[:, ::2], wg[:, :32], wu[:, :32], wd[:32]), ValueError),
            (lambda: lm.feed_forward(x, wg, wu, wd, out=x), ValueError),
            (lambda: lm.feed_forward(x, wg, wu, wd, out=out[:10]), ValueError),
            (lambda: lm.feed_forward(x.cpu(), wg, wu, wd), ValueError),
            (lambda: lm.feed_forward(x[:1].expand(20, 64), wg, wu, wd), lm.muon.MuonError),
            (lambda: lm.feed_forward(flat[1:1281].view(20, 64), wg, wu, wd), lm.muon.MuonError),
            (lambda: lm.feed_forward(x[:, :60], wg[:, :60], wu[:, :60], wd[:60]), lm.muon.MuonError),
            (lambda: lm.feed_forward(x, wg, wu, wd, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), lm.muon.MuonError),
            (lambda: lm.feed_forward_backward(dout, x, wg, wu, wd, None), TypeError),
            (lambda: lm.feed_forward_backward(dout, x, wg, wu, wd, kept[:, :10]), ValueError),
            (lambda: lm.feed_forward_backward(dout[:10], x, wg, wu, wd, kept), ValueError),
            (lambda: lm.feed_forward_backward(dout, x, wg, wu, wd, kept, dtype=torch.float16), TypeError),
            (lambda: lm.feed_forward_backward(dout, x, wg, wu, wd, kept, dx=dout), ValueError),
            (lambda: lm.feed_forward_backward(dout, x, wg, wu, wd, kept, dx=kept.view(-1)[:1280].view(20, 64)), ValueError)):
        with pytest.raises(error):
            fn()
    torch.cuda.synchronize()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    assert torch.equal(lm.feed_forward(x, wg, wu, wd, workspace=ws), lm.feed_forward(x, wg, wu, wd))
