"""Given outputs of the language-model operators: those that may be an input
hold the same bits as new ones, and those that share memory with what the
kernels still read are refused before any launch."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


def make(b, sq, sk, hq, hkv, d):
    g = torch.Generator().manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    return t(b, sq, hq, d), t(b, sk, hkv, d), t(b, sk, hkv, d), t(b, sq, hq, d)


@pytest.mark.parametrize("sq,sk,d,cap", [(1, 130, 64, 0.0), (1, 5000, 64, 0.0), (300, 300, 64, 0.0), (300, 300, 128, 20.0),
                                         (70, 4200, 128, 0.0)])
def test_outputs_in_place(lm, sq, sk, d, cap):
    q, k, v, dout = make(2, sq, sk, 4, 2, d)
    out, lse = lm.attention(q, k, v, softcap=cap)
    want = lm.attention_backward(dout, q, k, v, out, lse, softcap=cap)
    mine = q.clone()
    got, l2 = lm.attention(mine, k, v, softcap=cap, out=mine)
    assert got.data_ptr() == mine.data_ptr() and torch.equal(got, out) and torch.equal(l2, lse)
    dq, dk, dv = lm.attention_backward(dout, q, k, v, got, lse, softcap=cap, dq=got, dk=k, dv=v)
    assert (dq.data_ptr(), dk.data_ptr(), dv.data_ptr()) == (got.data_ptr(), k.data_ptr(), v.data_ptr())
    for x, y in zip((dq, dk, dv), want):
        assert torch.equal(x, y)


def test_norm_in_place(lm):
    q, k = (t.contiguous() for t in make(2, 9, 9, 4, 2, 64)[:2])
    table = torch.randn(20, 32, 2).cuda()
    want = lm.qk_norm_rope(q, k, table)
    got = lm.qk_norm_rope(q, k, table, q_out=q, k_out=k)
    assert got[0] is q and all(torch.equal(x, y) for x, y in zip(got, want))


def test_views_of_one_buffer_are_taken(lm):
    x = make(2, 150, 150, 8, 1, 64)[0]
    out = torch.empty_like(x)
    want = lm.attention(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:])[0]
    assert torch.equal(lm.attention(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], out=out[:, :, 4:])[0], want)
    # the output in the queries' place of the projection
    assert torch.equal(lm.attention(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], out=x[:, :, :4])[0], want)


def test_shared_memory_is_refused(lm):
    q, k, v, dout = make(2, 40, 40, 2, 2, 64)
    out, lse = lm.attention(q, k, v)
    table = torch.randn(40, 32, 2).cuda()
    emb, tok = torch.randn(40, 64).cuda(), torch.zeros(40, dtype=torch.long).cuda()
    flat = torch.zeros(3 * q.numel(), dtype=torch.bfloat16, device="cuda")
    part = lambda off: flat[off:off + q.numel()].view(q.shape)  # noqa: E731
    n = torch.full((160,), 40, dtype=torch.int32, device="cuda")
    back = lambda **kw: lm.attention_backward(dout, q, k, v, out, lse, **kw)  # noqa: E731
    for fn in (
            lambda: lm.attention(q, k, v, out=k), lambda: lm.attention(q, k, v, out=v),
            lambda: lm.attention(part(0), k, v, out=part(64)),
            lambda: lm.attention(q, k, v, out=part(0)[:, :, :1].expand_as(q)),
            lambda: lm.attention(q, k, v, out=part(0)[:1].expand_as(q)),
            lambda: lm.attention(q, k, v, lse=flat.view(torch.float32)[:160].view(2, 2, 40), out=part(0)),
            lambda: lm.attention(q, k, v, lengths=n[:2], lse=n.view(torch.float32).view(2, 2, 40)),
            lambda: back(dq=q), lambda: back(dq=dout), lambda: back(dq=k), lambda: back(dq=v), lambda: back(dk=q),
            lambda: back(dv=dout), lambda: back(dq=part(0), dk=part(64)), lambda: back(dk=part(0), dv=part(0)),
            lambda: lm.attention_backward(dout, q, k, v, part(0), lse, dq=part(64)),
            lambda: lm.attention_backward(dout, q, part(0), v, out, lse, dk=part(64)),
            lambda: lm.qk_norm_rope(q, k, table, q_out=k), lambda: lm.qk_norm_rope(q, k, table, k_out=q),
            lambda: lm.qk_norm_rope(part(0), k, table, q_out=part(64)),
            lambda: lm.qk_norm_rope(q, k, table, q_out=part(0), k_out=part(0)),
            lambda: lm.embedding(tok, emb, out=emb),
            lambda: lm.embedding_backward(emb, tok, 40, out=emb)):
        with pytest.raises(ValueError, match="share memory"):
            fn()
    torch.cuda.synchronize()
