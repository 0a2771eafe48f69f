"""The language-model operators' C ABI refuses misaligned side inputs (slopes,
masks, weights, table, positions) before it touches the HIP runtime: the kernels
load them as whole 4-byte values.  No GPU; no address here is dereferenced."""

import pytest

from .test_lm_abi import P, attn, lm, muon, qk  # noqa: F401


@pytest.mark.parametrize("name", ["slopes", "documents", "prefix", "lengths", "starts"])
def test_attention(lm, muon, name):  # noqa: F811
    for fn in (muon.lib.muon_attention, muon.lib.muon_attention_backward):
        for off in (1, 2, 3):
            assert fn(attn(lm, **{name: P + off}), P, 1 << 30, None) == muon.MUON_ERR_INVALID_ARG
            assert "aligned" in muon.lib.muon_last_error().decode()


def test_attention_documents_stride(lm, muon):  # noqa: F811
    for fn in (muon.lib.muon_attention, muon.lib.muon_attention_backward):
        assert fn(attn(lm, documents=P, documents_stride=-300), P, 1 << 30, None) == muon.MUON_ERR_INVALID_ARG
        assert "documents" in muon.lib.muon_last_error().decode()


@pytest.mark.parametrize("name", ["w0", "w1", "dw0", "dw1", "table", "positions"])
def test_norm_and_rotation(lm, muon, name):  # noqa: F811
    lib, kw = muon.lib, {name: P + 2}
    assert lib.muon_qk_norm_rope_backward(qk(lm, **kw), P, 1 << 30, None) == muon.MUON_ERR_INVALID_ARG
    assert "aligned" in lib.muon_last_error().decode()
    if not name.startswith("dw"):
        assert lib.muon_qk_norm_rope(qk(lm, **kw), None) == muon.MUON_ERR_INVALID_ARG
