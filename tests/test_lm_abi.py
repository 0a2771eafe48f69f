"""The language-model operators' C ABI without a GPU: libmuon.so exports what
include/muon_lm.h declares, sizes workspaces, and refuses invalid arguments
before it touches the HIP runtime (no kernel is launched here; every address
is made up and never dereferenced)."""

import os
import re

import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muon_lm.h")
P = 0x100000  # aligned to 256 bytes


@pytest.fixture(scope="module")
def lm():
    from newton_schulz_09_amd import lm as m
    return m


@pytest.fixture(scope="module")
def muon():
    from newton_schulz_09_amd import muon as m
    return m


def test_header_and_exports(lm, muon):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(muon_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(lm.EXPORTS)
    for n in names:
        assert hasattr(muon.lib, n), n
    for name, value in re.findall(r"#define MUON_(\w+_MAX_D) (\d+)", text):
        assert getattr(lm, name) == int(value)


ATTN = ["q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv",
        "qb", "qs", "qh", "kb", "ks", "kh", "vb", "vs", "vh", "ob", "os", "oh", "gb", "gs", "gh",
        "slopes", "documents", "documents_stride", "prefix", "lengths", "starts",
        "batch", "sq", "sk", "heads", "kv_heads", "d", "causal", "window", "scale", "softcap"]


def attn(lm, **kw):
    """Packed arguments of 2 sequences of 300 positions, 4 heads over 2, head size 64."""
    f = dict.fromkeys(ATTN, 0)
    f.update({n: P for n in ATTN[:9]})
    f.update(qb=300 * 256, qs=256, qh=64, kb=300 * 128, ks=128, kh=64, vb=300 * 128, vs=128, vh=64, ob=300 * 256,
             os=256, oh=64, gb=300 * 256, gs=256, gh=64, batch=2, sq=300, sk=300, heads=4, kv_heads=2, d=64, causal=1,
             scale=0.125, softcap=0.0)
    assert set(kw) <= set(f)
    f.update(kw)
    return lm._ATTN.pack(*[f[n] for n in ATTN])


def test_attention_workspace(lm, muon):
    size, back = muon.lib.muon_attention_workspace_size, muon.lib.muon_attention_backward_workspace_size
    assert size(attn(lm)) == 256
    assert back(attn(lm)) >= 2 * 4 * 300 * 2 * 4  # two float32 terms per query row
    assert size(attn(lm, documents=P)) >= 2 * 5 * 8
    # a step of generation over a long cache: partial results
    assert size(attn(lm, sq=1, sk=1 << 20)) > 2 * 4 * 2 * (64 + 2) * 4
    assert size(attn(lm, sk=0)) == 256 and size(attn(lm, batch=0)) == 256
    for bad in (dict(d=63), dict(d=136), dict(heads=3), dict(kv_heads=0), dict(batch=-1), dict(sq=1 << 29)):
        assert size(attn(lm, **bad)) == 0 and back(attn(lm, **bad)) == 0, bad
    assert size(None) == 0 and back(None) == 0


INVALID = [
    (dict(batch=-1), "negative"), (dict(sq=-1), "negative"), (dict(sk=-2), "negative"),
    (dict(heads=3), "multiple"), (dict(heads=0), "multiple"), (dict(kv_heads=0), "multiple"),
    (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(scale=1e-60), "scale"), (dict(softcap=-1.0), "softcap"),
    (dict(softcap=float("nan")), "softcap"), (dict(softcap=float("inf")), "softcap"), (dict(window=-1), "window"),
    (dict(q=0), "q is null"), (dict(k=0), "k is null"), (dict(v=0), "v is null"), (dict(out=0), "out is null"),
    (dict(lse=0), "lse"), (dict(lse=P + 2), "lse"), (dict(q=P + 8), "16 bytes"), (dict(out=P + 2), "16 bytes"),
    (dict(qs=260), "multiple of 8"), (dict(kh=4), "multiple of 8"), (dict(vb=-8), "multiple of 8"),
]
UNSUPPORTED = [dict(d=60), dict(d=0), dict(d=136), dict(sq=1 << 29), dict(sk=1 << 29), dict(ks=1 << 24),
               dict(batch=1 << 40), dict(batch=1 << 62, heads=1 << 62, kv_heads=1), dict(batch=1 << 20, heads=1 << 12, kv_heads=1)]


@pytest.mark.parametrize("kw,says", INVALID)
def test_attention_refuses(lm, muon, kw, says):
    lib = muon.lib
    for fn in (lib.muon_attention, lib.muon_attention_backward):
        assert fn(attn(lm, **kw), P, 1 << 30, None) == muon.MUON_ERR_INVALID_ARG
        assert says in lib.muon_last_error().decode()


@pytest.mark.parametrize("kw", UNSUPPORTED)
def test_attention_does_not_support(lm, muon, kw):
    for fn in (muon.lib.muon_attention, muon.lib.muon_attention_backward):
        assert fn(attn(lm, **kw), P, 1 << 30, None) == muon.MUON_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,says", [(dict(dout=0), "dout"), (dict(dq=0), "dq"), (dict(dk=0), "dk"), (dict(dv=0), "dv"),
                                     (dict(dq=P + 8), "dq"), (dict(dv=P + 8), "dv"), (dict(gs=4), "dout")])
def test_attention_backward_refuses(lm, muon, kw, says):
    assert muon.lib.muon_attention_backward(attn(lm, **kw), P, 1 << 30, None) == muon.MUON_ERR_INVALID_ARG
    assert says in muon.lib.muon_last_error().decode()


def test_attention_workspace_refusals_and_nothing_to_do(lm, muon):
    lib = muon.lib
    need = lib.muon_attention_backward_workspace_size(attn(lm))
    for ws, size in ((None, need), (P, need - 1), (P + 16, need)):
        assert lib.muon_attention_backward(attn(lm), ws, size, None) == muon.MUON_ERR_WORKSPACE
    assert lib.muon_attention(attn(lm), P, 255, None) == muon.MUON_ERR_WORKSPACE
    assert lib.muon_attention(None, P, 256, None) == muon.MUON_ERR_INVALID_ARG
    # nothing to compute: no launch, whatever the pointers
    empty = attn(lm, batch=0, q=0, k=0, v=0, out=0, lse=0, dout=0, dq=0, dk=0, dv=0)
    assert lib.muon_attention(empty, P, 256, None) == muon.MUON_OK
    assert lib.muon_attention_backward(empty, P, 256, None) == muon.MUON_OK
    assert lib.muon_attention(attn(lm, sq=0, q=0, out=0, lse=0), P, 256, None) == muon.MUON_OK


QK = ["x0", "x1", "out0", "out1", "dz0", "dz1", "w0", "w1", "dw0", "dw1",
      "x0b", "x0s", "x0h", "x1b", "x1s", "x1h", "z0b", "z0s", "z0h", "z1b", "z1s", "z1h", "heads0", "heads1",
      "table", "limit", "positions", "batch", "s", "d", "dtype", "eps"]


def qk(lm, **kw):
    f = dict.fromkeys(QK, 0)
    f.update({n: P for n in QK[:6]})
    f.update(x0b=5 * 256, x0s=256, x0h=64, x1b=5 * 128, x1s=128, x1h=64, z0b=5 * 256, z0s=256, z0h=64, z1b=5 * 128,
             z1s=128, z1h=64, heads0=4, heads1=2, table=P, limit=300, batch=2, s=5, d=64, dtype=1, eps=1e-6)
    assert set(kw) <= set(f)
    f.update(kw)
    return lm._QK.pack(*[f[n] for n in QK])


@pytest.mark.parametrize("kw,says", [
    (dict(batch=-1), "negative"), (dict(s=-1), "negative"), (dict(heads0=-1), "negative"), (dict(limit=-1), "negative"),
    (dict(dtype=2), "dtype"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(x0=0), "null"), (dict(out1=0), "null"), (dict(table=0), "table"), (dict(x1=P + 1), "aligned"),
    (dict(x0s=-8), "stride")])
def test_norm_and_rotation_refuses(lm, muon, kw, says):
    lib = muon.lib
    for st in (lib.muon_qk_norm_rope(qk(lm, **kw), None), lib.muon_qk_norm_rope_backward(qk(lm, **kw), P, 1 << 30, None)):
        assert st == muon.MUON_ERR_INVALID_ARG
        assert says in lib.muon_last_error().decode()


def test_norm_and_rotation_workspace_and_limits(lm, muon):
    lib = muon.lib
    size = lib.muon_qk_norm_rope_backward_workspace_size
    assert size(qk(lm)) >= 2 * 64 * 4
    for bad in (dict(d=63), dict(d=0), dict(d=514), dict(batch=1 << 29), dict(heads1=1 << 20), dict(limit=1 << 31)):
        assert size(qk(lm, **bad)) == 0
        assert lib.muon_qk_norm_rope(qk(lm, **bad), None) == muon.MUON_ERR_UNSUPPORTED
    assert lib.muon_qk_norm_rope_backward(qk(lm, dz0=0), P, 1 << 30, None) == muon.MUON_ERR_INVALID_ARG
    assert lib.muon_qk_norm_rope_backward(qk(lm, dw0=P), P, size(qk(lm)) - 1, None) == muon.MUON_ERR_WORKSPACE
    assert lib.muon_qk_norm_rope_backward(qk(lm, dw0=P), P + 4, 1 << 30, None) == muon.MUON_ERR_WORKSPACE
    assert lib.muon_qk_norm_rope(None, None) == muon.MUON_ERR_INVALID_ARG
    assert lib.muon_qk_norm_rope(qk(lm, batch=0, x0=0, x1=0, out0=0, out1=0, table=0), None) == muon.MUON_OK


def test_embedding_refuses(lm, muon):
    lib = muon.lib
    f32, bf16 = muon.MUON_F32, muon.MUON_BF16

    def both(tokens=P, token_bytes=8, src=P, src_type=f32, dst=P, dst_type=bf16, n=10, vocab=50, width=64, scale=1.0):
        need = 1 << 30
        a = lib.muon_embedding(tokens, token_bytes, src, src_type, dst, dst_type, n, vocab, width, scale, None)
        b = lib.muon_embedding_backward(tokens, token_bytes, src, src_type, dst, dst_type, n, vocab, width, scale, P,
                                        need, None)
        assert a == b
        return a

    inv = muon.MUON_ERR_INVALID_ARG
    for kw in (dict(tokens=None), dict(src=None), dict(dst=None), dict(token_bytes=2), dict(src_type=2), dict(dst_type=-1),
               dict(n=-1), dict(vocab=0), dict(width=0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(tokens=P + 4), dict(src=P + 2), dict(dst=P + 1)):
        assert both(**kw) == inv, kw
    for kw in (dict(n=1 << 31), dict(vocab=1 << 31), dict(width=(1 << 20) + 1)):
        assert both(**kw) == muon.MUON_ERR_UNSUPPORTED, kw
        full = dict(n=10, vocab=50, width=64, **{}) | kw
        assert lib.muon_embedding_backward_workspace_size(full["n"], full["vocab"], full["width"]) == 0
    assert lib.muon_embedding(None, 8, None, f32, None, f32, 0, 50, 64, 1.0, None) == muon.MUON_OK
    need = lib.muon_embedding_backward_workspace_size(10, 50, 64)
    assert need >= 2 * 10 * 4 + 51 * 4 + 2 * 64 * 4
    for ws, size in ((None, need), (P, need - 1), (P + 128, need)):
        assert lib.muon_embedding_backward(P, 8, P, f32, P, f32, 10, 50, 64, 1.0, ws, size, None) == muon.MUON_ERR_WORKSPACE


def test_binding_refuses_cpu_tensors_and_other_things(lm):
    import torch
    t = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    for fn in (lambda: lm.attention(t, t, t), lambda: lm.attention_backward(t, t, t, t, t, t),
               lambda: lm.qk_norm_rope(t, t, torch.zeros(4, 32, 2)), lambda: lm.embedding(torch.zeros(3, dtype=torch.long), t),
               lambda: lm.embedding_backward(t, torch.zeros(1, dtype=torch.long), 4)):
        with pytest.raises(ValueError):
            fn()
    for fn in (lambda: lm.attention(None, t, t), lambda: lm.attention_backward(t, None, t, t, t, t),
               lambda: lm.qk_norm_rope(3, t, t), lambda: lm.qk_norm_rope_backward(t, t, 3, t, t),
               lambda: lm.embedding([1], t), lambda: lm.embedding_backward(t, [1], 4)):
        with pytest.raises(TypeError):
            fn()
