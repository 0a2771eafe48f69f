"""The C ABI of the decoder layer's operators without a GPU: workspaces, refused
arguments (no kernel is launched; every address is made up and never
dereferenced), and the generator's and the gradients' definitions."""

import math

import pytest
import torch

from tests import layer_reference as ref

P = 0x100000  # aligned to 256 bytes


@pytest.fixture(scope="module")
def lm():
    from newton_schulz_09_amd import lm as m
    return m


@pytest.fixture(scope="module")
def muon():
    from newton_schulz_09_amd import muon as m
    return m


# ------------------------------------------------------------ feed-forward

FFN = ["x", "w_gate", "w_up", "w_down", "out", "kept", "dout", "dx", "dw_gate", "dw_up", "dw_down",
       "x_stride", "w_stride", "w_down_stride", "dout_stride", "tokens", "width", "hidden", "activation", "dw_type"]


def ffn(lm, **kw):
    f = dict.fromkeys(FFN, P)
    f.update(x_stride=64, w_stride=64, w_down_stride=136, dout_stride=64, tokens=40, width=64, hidden=136, activation=0,
             dw_type=1)
    assert set(kw) <= set(f)
    f.update(kw)
    return lm._FFN.pack(*[f[n] for n in FFN])


FFN_INVALID = [
    (dict(tokens=-1), "negative"), (dict(activation=4), "activation"), (dict(activation=-1), "activation"),
    (dict(x=0), "x is null"), (dict(w_gate=0), "w_gate"), (dict(w_up=0), "w_up"), (dict(w_down=0), "w_down"),
    (dict(x=P + 8), "16 bytes"), (dict(w_down=P + 2), "16 bytes"), (dict(x_stride=68), "multiple of 8"),
    (dict(x_stride=56), "multiple of 8"), (dict(x_stride=0), "multiple of 8"), (dict(w_stride=-64), "multiple of 8"),
    (dict(w_down_stride=128), "multiple of 8")]
FFN_UNSUPPORTED = [dict(width=60), dict(hidden=4), dict(width=0), dict(hidden=-8), dict(width=1 << 21), dict(tokens=1 << 29),
                   dict(x_stride=1 << 21), dict(tokens=(1 << 29) - 1, width=(1 << 21) - 8)]


@pytest.mark.parametrize("kw,says", FFN_INVALID)
def test_feed_forward_refuses(lm, muon, kw, says):
    for fn in (muon.lib.muon_feed_forward, muon.lib.muon_feed_forward_backward):
        assert fn(ffn(lm, **kw), P, 1 << 40, None) == muon.MUON_ERR_INVALID_ARG
        assert says in muon.lib.muon_last_error().decode()


@pytest.mark.parametrize("kw", FFN_UNSUPPORTED)
def test_feed_forward_does_not_support(lm, muon, kw):
    for fn in (muon.lib.muon_feed_forward, muon.lib.muon_feed_forward_backward):
        assert fn(ffn(lm, **kw), P, 1 << 40, None) == muon.MUON_ERR_UNSUPPORTED
    if "x_stride" not in kw:
        assert muon.lib.muon_feed_forward_workspace_size(ffn(lm, **kw)) == 0
        assert muon.lib.muon_feed_forward_backward_workspace_size(ffn(lm, **kw)) == 0


def test_feed_forward_other_refusals(lm, muon):
    lib = muon.lib
    inv = muon.MUON_ERR_INVALID_ARG
    assert lib.muon_feed_forward(ffn(lm, out=0), P, 1 << 40, None) == inv
    assert lib.muon_feed_forward(ffn(lm, kept=P + 8), P, 1 << 40, None) == inv
    for kw in (dict(dout=0), dict(dx=0), dict(kept=0), dict(dw_gate=0), dict(dw_up=P + 4), dict(dw_down=0), dict(dw_type=2),
               dict(dout_stride=8)):
        assert lib.muon_feed_forward_backward(ffn(lm, **kw), P, 1 << 40, None) == inv, kw
    for fn, size in ((lib.muon_feed_forward, lib.muon_feed_forward_workspace_size),
                     (lib.muon_feed_forward_backward, lib.muon_feed_forward_backward_workspace_size)):
        kept = {"kept": 0} if fn is lib.muon_feed_forward else {}  # (where it is given, it holds the hidden values)
        need = size(ffn(lm, **kept))
        assert need >= 40 * 136 * 2 and size(ffn(lm)) >= 256
        for ws, n in ((None, need), (P, need - 1), (P + 16, need)):
            assert fn(ffn(lm, **kept), ws, n, None) == muon.MUON_ERR_WORKSPACE
        assert fn(None, P, 256, None) == inv and size(None) == 0
    # no tokens: nothing to compute, whatever their pointers
    assert lib.muon_feed_forward(ffn(lm, tokens=0, x=0, out=0, kept=0), P, 256, None) == muon.MUON_OK


# ---------------------------------------------------- norms around a block

RESID = ["x", "y", "gate", "residual_scale", "post_weight", "pre_weight", "x_out", "z", "dz", "dx_out", "dx", "dy", "dgate",
         "dresidual_scale", "dpost_weight", "dpre_weight", "x_stride", "y_stride", "gate_stride", "x_out_stride", "dz_stride",
         "dx_out_stride", "batch", "s", "width", "stream_type", "block_type", "has_block", "post", "gate_kind", "eps", "p", "seed",
         "offset", "state"]


def resid(lm, **kw):
    f = dict.fromkeys(RESID, P)
    f.update({n: 96 for n in RESID if n.endswith("_stride")})
    f.update(batch=2, s=5, width=96, stream_type=1, block_type=1, has_block=1, post=1, gate_kind=3, eps=1e-6, p=0.1, seed=1,
             offset=0, state=0)
    assert set(kw) <= set(f)
    f.update(kw)
    return lm._RESID.pack(*[f[n] for n in RESID])


RESID_INVALID = [
    (dict(batch=-1), "negative"), (dict(s=-1), "negative"), (dict(stream_type=2), "dtype"), (dict(block_type=-1), "dtype"),
    (dict(gate_kind=4), "gate_kind"), (dict(eps=-1.0), "eps"), (dict(eps=math.nan), "eps"), (dict(eps=math.inf), "eps"),
    (dict(p=-0.1), "p must"), (dict(p=1.5), "p must"), (dict(p=math.nan), "p must"), (dict(state=P + 4), "state"),
    (dict(y=0), "y is null"), (dict(y=P + 1), "y is null"), (dict(y_stride=-96), "y is null"), (dict(gate=0), "gate is null"),
    (dict(gate_kind=1, gate=0), "gate is null"), (dict(gate_kind=2, gate=0), "gate is null"), (dict(gate_kind=1, gate=P + 2), "4 bytes"),
    (dict(has_block=0), "without a block"), (dict(has_block=0, gate_kind=0, post=0), "without a block"),
    (dict(post=0), "post norm without"), (dict(pre_weight=P + 2), "4 bytes"), (dict(residual_scale=P + 1), "4 bytes")]


@pytest.mark.parametrize("kw,says", RESID_INVALID)
def test_norms_refuse(lm, muon, kw, says):
    lib = muon.lib
    for st in (lib.muon_residual_norm(resid(lm, **kw), None), lib.muon_residual_norm_backward(resid(lm, **kw), P, 1 << 40, None)):
        assert st == muon.MUON_ERR_INVALID_ARG
        assert says in lib.muon_last_error().decode()


def test_norms_other_refusals(lm, muon):
    lib = muon.lib
    assert lib.muon_residual_norm(resid(lm, x=0), None) == muon.MUON_ERR_INVALID_ARG
    assert lib.muon_residual_norm(resid(lm, z=P + 1), None) == muon.MUON_ERR_INVALID_ARG
    for kw in (dict(x_out=0), dict(dz=0), dict(dx=0), dict(dy=0), dict(dgate=0), dict(x=0), dict(dx_out=P + 1),
               dict(gate_kind=1, dgate=0), dict(gate_kind=2, dgate=0), dict(residual_scale=0), dict(dpre_weight=P + 2),
               dict(dz_stride=-1)):
        assert lib.muon_residual_norm_backward(resid(lm, **kw), P, 1 << 40, None) == muon.MUON_ERR_INVALID_ARG, kw
    size = lib.muon_residual_norm_backward_workspace_size
    for kw in (dict(width=0), dict(width=8193), dict(batch=1 << 29), dict(s=1 << 29), dict(batch=(1 << 20) + 1, gate_kind=2),
               dict(block_type=0)):
        assert lib.muon_residual_norm(resid(lm, **kw), None) == muon.MUON_ERR_UNSUPPORTED, kw
        assert lib.muon_residual_norm_backward(resid(lm, **kw), P, 1 << 40, None) == muon.MUON_ERR_UNSUPPORTED, kw
        assert size(resid(lm, **kw)) == 0
    need = size(resid(lm))
    assert need >= 4 * 96 * 4
    for ws, n in ((None, need), (P, need - 1), (P + 16, need)):
        assert lib.muon_residual_norm_backward(resid(lm), ws, n, None) == muon.MUON_ERR_WORKSPACE
    assert lib.muon_residual_norm(None, None) == lib.muon_residual_norm_backward(None, P, 256, None) == muon.MUON_ERR_INVALID_ARG
    assert lib.muon_residual_norm(resid(lm, batch=0, x=0, y=0, gate=0, x_out=0, z=0), None) == muon.MUON_OK


def test_dropout_refuses(muon):
    fn = muon.lib.muon_dropout

    def call(x=P, out=P, n=10, dtype=0, p=0.5, state=None):
        return fn(x, out, n, dtype, p, 1, 0, state, None)

    for kw in (dict(x=None), dict(out=None), dict(x=P + 2), dict(out=P + 1), dict(n=-1), dict(dtype=2), dict(p=-0.1), dict(p=1.1),
               dict(p=math.nan), dict(state=P + 4)):
        assert call(**kw) == muon.MUON_ERR_INVALID_ARG, kw
    assert call(n=(1 << 41) + 1) == muon.MUON_ERR_UNSUPPORTED
    assert call(n=0, x=None, out=None) == muon.MUON_OK


def test_binding_refuses_cpu_tensors_and_other_things(lm):
    t, v = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    for fn in (lambda: lm.dropout(t, 0.1, 3), lambda: lm.residual_norm(t, t), lambda: lm.residual_norm_backward(t, t, t, t),
               lambda: lm.feed_forward(t, t, t, t), lambda: lm.feed_forward_backward(t, t, t, t, t, t)):
        with pytest.raises(ValueError):
            fn()
    for fn in (lambda: lm.dropout([1], 0.1, 3), lambda: lm.residual_norm(None, t), lambda: lm.residual_norm_backward(t, t, 3),
               lambda: lm.feed_forward(v.tolist(), t, t, t), lambda: lm.feed_forward_backward(t, 3, t, t, t, t)):
        with pytest.raises(TypeError):
            fn()


# ------------------------------------------------------------- definitions

def test_the_generators_known_answers():
    """Philox4x32-10's published answers for the counter and key zero (whose
    other words the layout here leaves zero), and the counter's carry."""
    assert ref.philox(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox(0, 1 << 32) != ref.philox(0, 0) != ref.philox(1 << 32, 0)
    assert ref.bits(0, 0)[:2] == [0xE8D5, 0x6627]


def test_the_gradients_definitions_against_differences():
    """Central differences in float64: the formulas the kernels are held to."""
    g = torch.Generator().manual_seed(3)
    t = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    h = 1e-5

    def slope(f, args, k, d):
        up, down = ([a + (s * h * d if i == k else 0) for i, a in enumerate(args)] for s in (1, -1))
        return float((f(*up) - f(*down)) / (2 * h))

    for name in ref.SLOPE:
        args = [t(5, 16), t(24, 16), t(24, 16), t(16, 24)]
        dout = t(5, 16)
        res, _ = ref.feed_forward(*args, name, dout)
        f = lambda *a: (ref.feed_forward(*a, name)[0]["out"] * dout).sum()  # noqa: E731
        for k, key in enumerate(("dx", "dwg", "dwu", "dwd")):
            d = t(*args[k].shape)
            want = float((res[key] * d).sum())
            assert abs(slope(f, args, k, d) - want) < 1e-6 * (1 + abs(want)), (name, key)
    for gate in ((16,), (2, 16), (2, 3, 16), None):
        for post in (True, False):
            factor = (t(2, 3, 16) > 0).double() * 1.5
            args = [t(2, 3, 16), t(2, 3, 16), t(*gate) if gate else None, t(16), t(16) if post else None, t(16)]
            dz, dxo = t(2, 3, 16), t(2, 3, 16)

            def f(*a):
                r = ref.residual_norm(*a, post=post, factor=factor)[0]
                return (r["z"] * dz).sum() + (r["x_out"] * dxo).sum()

            def fill(*some):
                it = iter(some)
                return f(*[None if a is None else next(it) for a in args])

            xo = ref.residual_norm(*args, post=post, factor=factor)[0]["x_out"]
            res, _ = ref.residual_norm(*args, post=post, factor=factor, xo=xo, dz=dz, dxo=dxo)
            there = [a for a in args if a is not None]
            keys = [k for k, a in zip(("dx", "dy", "dgate", "dscale", "dpostw", "dprew"), args) if a is not None]
            for k, key in enumerate(keys):
                d = t(*there[k].shape)
                want = float((res[key] * d).sum())
                assert abs(slope(fill, there, k, d) - want) < 1e-6 * (1 + abs(want)), (gate, post, key)
