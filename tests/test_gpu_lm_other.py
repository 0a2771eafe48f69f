"""The norm and rotation of query and key heads and the embedding, with their
gradients, on the GPU against float64 definitions."""

import math

import pytest
import torch

from . import lm_reference as ref

pytestmark = pytest.mark.gpu
F32, BF = ref.F32, ref.BF


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


def table(d, limit=300):
    a = torch.arange(limit, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    return torch.stack([a.cos(), a.sin()], -1).float().cuda()


def half_step(dtype):
    return BF if dtype == torch.bfloat16 else F32


def qk_inputs(b, s, hq, hkv, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda *sh: torch.randn(*sh, generator=g)  # noqa: E731
    qkv = t(b, s, hq + 2 * hkv, d).to(dtype).cuda()
    return (qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], (1 + 0.2 * t(d)).cuda(), (1 + 0.2 * t(d)).cuda(),
            t(b, s, hq, d).to(dtype).cuda(), t(b, s, hkv, d).to(dtype).cuda(),
            torch.randint(0, 300, (b, s), generator=g).int().cuda())


def check_qk(lm, q, k, qw, kw, dq, dk, pos, tab, weights, eps=1e-6):
    print(f"norm and rotation {tuple(q.shape)} {tuple(k.shape)} {q.dtype} weights {weights}", flush=True)
    dtype, d = q.dtype, q.shape[-1]
    wq, wk = (qw, kw) if weights else (None, None)
    got = lm.qk_norm_rope(q, k, tab, positions=pos, q_weight=wq, k_weight=wk, eps=eps)
    grad = lm.qk_norm_rope_backward(dq, dk, q, k, tab, positions=pos, q_weight=wq, k_weight=wk, eps=eps)
    torch.cuda.synchronize()
    at = pos if pos is not None else torch.arange(q.shape[1]).expand(q.shape[:2])
    for n, (x, w, dz) in enumerate(((q, wq, dq), (k, wk, dk))):
        leaf = x.detach().cpu().double().requires_grad_()
        wd = None if w is None else w.cpu().double().requires_grad_()
        xs = leaf / (leaf.square().mean(-1, keepdim=True) + eps).sqrt()
        y = xs if wd is None else xs * wd
        cs = tab.cpu().double()[at.cpu().long()][:, :, None]
        a, b = y[..., :d // 2], y[..., d // 2:]
        z = torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]], -1)
        z.backward(dz.cpu().double())
        # float32: the sum of d squares, then a dozen roundings, relative to
        # the halves' magnitudes; one rounding to the type
        e = (d + 16) * F32
        mag = torch.maximum(a.abs() + b.abs(), torch.zeros(()).double()).detach()
        ref.close(got[n], z.detach(), half_step(dtype) * z.abs().detach() + (e + half_step(dtype) * e) * torch.cat([mag, mag], -1), "qk"[n])
        t1, t2 = dz.cpu().double()[..., :d // 2].abs(), dz.cpu().double()[..., d // 2:].abs()
        tm = torch.cat([t1 + t2, t1 + t2], -1) * (1.0 if w is None else w.cpu().double().abs())
        xs = xs.detach()
        r = (leaf.square().mean(-1, keepdim=True) + eps).rsqrt().detach()
        bound = r * (tm + xs.abs() * (tm * xs.abs()).mean(-1, keepdim=True)) * 3 * e
        ref.close(grad[n], leaf.grad, half_step(dtype) * leaf.grad.abs() + 2 * bound, "d" + "qk"[n])
        if w is not None:
            rows = x[..., 0].numel()
            tw = (torch.cat([t1 + t2, t1 + t2], -1) * xs.abs()).sum((0, 1, 2))
            ref.close(grad[2 + n], wd.grad, (e + (rows + 8) * F32) * tw, f"d{'qk'[n]}w")
        else:
            assert grad[2 + n] is None


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 64), (2, 7, 6, 2, 64), (1, 33, 4, 1, 80), (3, 5, 12, 3, 96),
                                   (1, 129, 8, 8, 128), (2, 3, 2, 1, 2), (1, 4, 3, 1, 10), (1, 5, 2, 2, 256),
                                   (1, 3, 2, 1, 512), (1, 3, 2, 1, 390), (1, 40, 24, 1, 16)])
def test_norm_and_rotation(lm, shape, dtype, weights):
    check_qk(lm, *qk_inputs(*shape, dtype), table(shape[-1]), weights)


def test_norm_layouts(lm):
    q, k, qw, kw, dq, dk, pos = qk_inputs(2, 9, 4, 2, 64, torch.bfloat16)
    check_qk(lm, q, k, qw, kw, dq, dk, None, table(64), True)  # positions 0 .. s - 1
    base = torch.randn(2, 9, 6, 67).bfloat16().cuda()          # rows that are not aligned
    check_qk(lm, base[:, :, :4, 1:65], base[:, :, 4:, 1:65], qw, kw, dq, dk, pos, table(64), True)
    t = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    check_qk(lm, t(q), t(k), qw, kw, t(dq), t(dk), pos, table(64), True)
    check_qk(lm, q, k, qw, kw, dq[:, :, :1].expand_as(q), dk, pos, table(64), True)


def test_norm_edges(lm):
    q, k, qw, kw, dq, dk, pos = qk_inputs(2, 5, 3, 1, 64, torch.float32)
    q, k = q.clone(), k.clone()
    q[0] = 0  # a head of zeros: only eps is left
    check_qk(lm, q, k, qw, kw, dq, dk, pos, table(64), True)
    pos[0, 0], pos[1, 4] = -1, 300
    out, _ = lm.qk_norm_rope(q, k, table(64), positions=pos)
    bad = torch.isnan(out).all(-1).all(-1).cpu()
    want = torch.zeros(2, 5, dtype=torch.bool)
    want[0, 0] = want[1, 4] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(out).any(-1).any(-1).cpu(), want)
    for b, s in ((0, 5), (2, 0)):
        q, k, qw, kw, dq, dk, pos = qk_inputs(b, s, 3, 1, 64, torch.float32)
        assert lm.qk_norm_rope(q, k, table(64))[0].shape == (b, s, 3, 64)
        g = lm.qk_norm_rope_backward(dq, dk, q, k, table(64), q_weight=qw, k_weight=kw)
        assert g[0].numel() == 0 and not g[2].any() and not g[3].any()


def test_norm_many_rows_same_bits(lm):
    q, k, qw, kw, dq, dk, pos = qk_inputs(8, 700, 6, 2, 64, torch.bfloat16)
    check_qk(lm, q, k, qw, kw, dq, dk, pos, table(64), True)
    a = lm.qk_norm_rope_backward(dq, dk, q, k, table(64), positions=pos, q_weight=qw, k_weight=kw)
    b = lm.qk_norm_rope_backward(dq, dk, q, k, table(64), positions=pos, q_weight=qw, k_weight=kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def check_embed(lm, tokens, vocab, width, ttype, otype, scale):
    print(f"embedding {tuple(tokens.shape)} of {vocab} x {width} {ttype} {otype}", flush=True)
    g = torch.Generator().manual_seed(1)
    tab = torch.randn(vocab, width, generator=g).to(ttype).cuda()
    out = lm.embedding(tokens, tab, scale=scale, dtype=otype)
    torch.cuda.synchronize()
    s = torch.tensor(scale, dtype=torch.float32).double()  # the factor is float32
    want = tab.cpu().double()[tokens.cpu().long()] * s
    ref.close(out, want, (half_step(otype) + 2 * F32) * want.abs(), "rows")
    dout = torch.randn(*tokens.shape, width, generator=g).to(otype).cuda()
    grad = lm.embedding_backward(dout, tokens, vocab, scale=scale, dtype=ttype)
    torch.cuda.synchronize()
    flat, d = tokens.cpu().long().reshape(-1), dout.cpu().double().reshape(-1, width)
    want = torch.zeros(vocab, width, dtype=torch.float64).index_add_(0, flat, d) * s
    mag = torch.zeros(vocab, width, dtype=torch.float64).index_add_(0, flat, d.abs()) * abs(s)
    n = torch.bincount(flat, minlength=vocab)[:, None].double()
    ref.close(grad, want, half_step(ttype) * want.abs() + (n + 2) * F32 * (1 + half_step(ttype)) * mag, "gradient")
    again = lm.embedding_backward(dout, tokens, vocab, scale=scale, dtype=ttype)
    assert torch.equal(grad, again)


@pytest.mark.parametrize("ttype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("otype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,width", [(1, 1, 8), (1, 300, 64), (63, 7, 100), (64, 1, 64), (65, 1000, 13),
                                           (1000, 3, 96), (4097, 50257, 16), (777, 513, 1600), (300, 40, 2056),
                                           (129, 128, 1)])
def test_embedding(lm, n, vocab, width, ttype, otype):
    g = torch.Generator().manual_seed(n)
    check_embed(lm, torch.randint(0, vocab, (n,), generator=g).cuda(), vocab, width, ttype, otype, math.sqrt(width))


def test_embedding_token_patterns(lm):
    f = torch.float32
    check_embed(lm, torch.full((3000,), 5).cuda(), 11, 64, f, f, 1.0)                       # one token
    check_embed(lm, torch.arange(640).flip(0).cuda(), 640, 64, f, f, -2.0)                  # each once
    check_embed(lm, torch.arange(64).repeat_interleave(64).cuda(), 64, 64, f, f, 1.0)       # whole windows
    check_embed(lm, torch.arange(40).repeat(50).int().reshape(4, 500).cuda(), 41, 24, f, f, 1.0)
    g = torch.Generator().manual_seed(2)
    z = (torch.rand(20000, generator=g, dtype=torch.float64) * math.log(140001)).exp().long() - 1
    check_embed(lm, z.cuda(), 140000, 8, f, torch.bfloat16, 3.0)                            # long-tailed, wide table


def test_embedding_tokens_outside_the_table(lm):
    t = torch.tensor([0, -1, 3, 4, 2 ** 40, 3, -2 ** 62]).cuda()
    tab = torch.randn(4, 16).cuda()
    out = lm.embedding(t, tab)
    bad = torch.tensor([False, True, False, True, True, False, True])
    assert torch.equal(torch.isnan(out).all(-1).cpu(), bad)
    assert torch.equal(out[~bad.cuda()], tab[t[~bad.cuda()]])
    dout = torch.ones(7, 16).cuda()
    assert torch.equal(lm.embedding_backward(dout, t, 4)[:, 0].cpu(), torch.tensor([1.0, 0.0, 0.0, 2.0]))


def test_embedding_empty_and_unaligned(lm):
    tab = torch.randn(5, 16).cuda()
    t = torch.zeros(0, dtype=torch.long).cuda()
    assert lm.embedding(t, tab).shape == (0, 16)
    assert not lm.embedding_backward(torch.zeros(0, 16).cuda(), t, 5).any()
    flat = torch.randn(5 * 16 + 1).cuda()[1:].view(5, 16)  # four bytes off
    t = torch.tensor([4, 0, 4]).cuda()
    assert torch.equal(lm.embedding(t, flat), flat[t])
    assert torch.equal(lm.embedding_backward(flat[:3], t, 5)[4], flat[0] + flat[2])


def test_graph(lm):
    q, k, qw, kw, dq, dk, pos = qk_inputs(2, 50, 4, 2, 64, torch.bfloat16)
    tab, emb = table(64), torch.randn(300, 64).cuda()
    tok = torch.randint(0, 300, (500,)).cuda()
    dout = torch.randn(500, 64).cuda()

    def run():
        return (*lm.qk_norm_rope(q, k, tab, pos, qw, kw), *lm.qk_norm_rope_backward(dq, dk, q, k, tab, pos, qw, kw),
                lm.embedding(tok, emb), lm.embedding_backward(dout, tok, 300))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in range(3):
        q.normal_()
        dq.normal_()
        tok.random_(0, 300)
        dout.normal_()
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), seed


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2000])
@pytest.mark.parametrize("vocab,width", [(1, 64), (33, 8), (300, 2064), (8200, 96), (700, 7)])
def test_embedding_gradient_at_the_borders_of_its_variants(lm, n, vocab, width):
    g = torch.Generator().manual_seed(n + vocab)
    tokens = (torch.rand(n, generator=g, dtype=torch.float64) ** 3 * vocab).long()
    check_embed(lm, tokens.cuda(), vocab, width, torch.bfloat16, torch.bfloat16, 1.0)
    check_embed(lm, tokens.int().cuda(), vocab, width, torch.float32, torch.bfloat16, 0.5)


@pytest.mark.parametrize("n", [5, 3000])
def test_embedding_offsets_past_32_bits(lm, n):
    """A table of 2.3e9 elements (4.6 GB)."""
    vocab, width = 70000, 32768
    table = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(6)
    rows = torch.tensor([0, 1, 65535, 65536, 65537, 69999]).cuda()
    table[rows] = torch.randn(6, width, generator=g).bfloat16().cuda()
    tokens = rows[torch.randint(0, 6, (n,), generator=g).cuda()]
    assert torch.equal(lm.embedding(tokens, table), table[tokens])
    dout = torch.randint(-3, 4, (n, width), generator=g).bfloat16().cuda()  # sums of whole numbers are exact
    table.fill_(7.0)
    lm.embedding_backward(dout, tokens, vocab, dtype=torch.bfloat16, out=table)
    for r in rows.tolist():
        want = dout[tokens == r].float().sum(0).bfloat16()
        assert torch.equal(table[r], want), r
    assert int((table != 0).any(1).sum()) <= 6


def test_norm_offsets_past_32_bits(lm):
    b, s, step = 3, 9, 2 ** 31
    flat = torch.empty((b - 1) * step + s * 128, dtype=torch.bfloat16, device="cuda")
    q, k, qw, kw, dq, dk, pos = qk_inputs(b, s, 2, 1, 64, torch.bfloat16)
    x = flat.as_strided((b, s, 2, 64), (step, 128, 64, 1))
    x.copy_(q)
    check_qk(lm, x, k, qw, kw, dq, dk, pos, table(64), True)
