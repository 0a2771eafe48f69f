"""The feed-forward block's activations over their whole range, one gate at a
time, against the definition in float64.

Every product here has one term that is not zero, so the gate, the up projection
and the gradient of the hidden values reach the activation exactly, and what is
left are the steps of the activation and one rounding to bfloat16."""

import math

import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu
B = torch.bfloat16
NAMES = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


def run(lm, gates, name, n):
    """(h without kept values, h, gradients of gate and up projection) of bfloat16
    gates (a multiple of 8 of them), for an up projection and a gradient of ones."""
    hidden = len(gates)
    x = torch.zeros(n, 8, dtype=B)
    x[:, 0] = 1
    wg = torch.zeros(hidden, 8, dtype=B)
    wg[:, 0] = gates
    wu = torch.zeros(hidden, 8, dtype=B)
    wu[:, 0] = 1
    x, wg, wu = x.cuda(), wg.cuda(), wu.cuda()
    one = torch.eye(hidden, dtype=B)  # the result's columns are the hidden values
    got = []
    for first in range(0, hidden, 8):
        got.append(lm.feed_forward(x, wg, wu, one[first:first + 8].contiguous().cuda(), activation=name)[-1])
    wd = torch.zeros(8, hidden, dtype=B)
    wd[0] = 1
    wd = wd.cuda()
    out, kept = lm.feed_forward(x, wg, wu, wd, activation=name, keep=True)
    dout = torch.zeros(n, 8, dtype=B)
    dout[-1, 0] = 1  # the last token's alone
    _, dwg, dwu, _ = lm.feed_forward_backward(dout.cuda(), x, wg, wu, wd, kept, activation=name, dtype=torch.float32)
    return torch.cat(got), kept[2, -1], dwg[:, 0], dwu[:, 0]


def definition(name, g):
    """act(g) and its derivative, without the cancellation of 1 + tanh."""
    g = g.double()
    if name in ("relu", "gelu"):
        return ref.act(name, g)
    k, c = (1.0, 0.0) if name == "silu" else (2 * math.sqrt(2 / math.pi), 0.044715)
    v, slope = k * (g + c * g ** 3), k * (1 + 3 * c * g * g)
    s = torch.sigmoid(v)
    return g * s, s + g * s * torch.sigmoid(-v) * slope


def relative(got, want, g, what):
    """Within one rounding to bfloat16 (2^-8) and what float32 leaves: the argument
    of the exponential, at most 90 for values that float32 holds, is off by
    three roundings of 2^-24 each, so the exponential by 300 2^-24 < 2^-15; the other steps are a
    dozen roundings, whose sum cancels by less than 16 at these gates.  Values
    below 2^-120 may be lost."""
    got = got.double().cpu()
    over = (got - want).abs() - (2.0 ** -8 + 2.0 ** -15 + 200 * 2.0 ** -24) * want.abs() - 2.0 ** -120
    assert torch.isfinite(got).all() and (over <= 0).all(), (what, g[over > 0].tolist()[:8], got[over > 0].tolist()[:8],
                                                            want[over > 0].tolist()[:8])


# the kernels of a few tokens, and tiles
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("name", NAMES)
def test_tails(lm, name, n):
    """Gates from -12 to -3.5, where act(gate) falls to 1e-32, and their mirror images."""
    g = torch.linspace(3.5, 12.0, 252, dtype=torch.float64).to(B)
    g = torch.cat([-g, g, torch.tensor([-0.01, 0.01, -1e-3, 1e-3, -1e-20, 1e-20, 0.5, 1.0], dtype=torch.float64).to(B)])
    a, da = definition(name, g)
    few, h, dg, du = run(lm, g, name, n)
    for got, want, what in ((few, a, "out"), (h, a, "h"), (du, a, "du"), (dg, da, "dg")):
        relative(got, want, g, (name, n, what))


@pytest.mark.parametrize("name", NAMES)
def test_large_gates(lm, name):
    """Finite gates of any size."""
    g = torch.tensor([2.0 ** e for e in (5, 10, 20, 40, 60, 62, 63, 64, 65, 66, 70, 80, 100, 120, 126, 127)], dtype=torch.float64).to(B)
    g = torch.cat([g, -g])
    few, h, dg, du = run(lm, g, name, 3)
    a, da = definition(name, g)
    for got, want, what in ((few, a, "out"), (h, a, "h"), (du, a, "du"), (dg, da, "dg")):
        relative(got, want, g, (name, what))
