"""What no query sees, and queries that see nothing, may hold NaN: attention and
its gradients against the float64 definition without them."""

import pytest
import torch

from . import lm_bounds
from . import lm_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


def ints(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def check(lm, b, sq, sk, hq, hkv, d, softcap=0.0, keys=True, **mask):
    """NaN at the keys past the last seen one (keys) and in queries that see none."""
    print(f"attention {b} x {sq} over {sk}, {hq} heads of {d} over {hkv}, {sorted(mask)}", flush=True)
    g = torch.Generator().manual_seed(sq + sk)
    q, k, v, dout = (torch.randn(*s, generator=g).bfloat16().cuda()
                     for s in ((b, sq, hq, d), (b, sk, hkv, d), (b, sk, hkv, d), (b, sq, hq, d)))
    vis, pos = ref.visible(b, sq, sk, **{n: t.cpu() if torch.is_tensor(t) else t for n, t in mask.items()})
    for n in range(b):
        seen = vis[n].any(0).nonzero()
        last = int(seen[-1]) + 1 if len(seen) else 0
        if keys:
            k[n, last:] = float("nan")
            v[n, last:] = float("inf")
        blind = (~vis[n].any(1)).cuda()
        q[n, blind] = float("nan")
        dout[n, blind] = float("nan")
    want, tol = lm_bounds.attention(q, k, v, dout, vis, pos, softcap=softcap)
    out, lse = lm.attention(q, k, v, softcap=softcap, **mask)
    grads = lm.attention_backward(dout, q, k, v, out, lse, softcap=softcap, **mask)
    torch.cuda.synchronize()
    for t, name in zip((out, lse, *grads), ("out", "lse", "dq", "dk", "dv")):
        ref.close(t, want[name], tol[name], name)


@pytest.mark.parametrize("sq", [1, 5, 70, 200])
@pytest.mark.parametrize("d,cap", [(64, 0.0), (128, 0.0), (128, 20.0), (80, 0.0)])
def test_caches_past_their_last_position(lm, sq, d, cap):
    check(lm, 3, sq, 500, 4, 2, d, softcap=cap, starts=ints(0, 131, 499 - sq))
    check(lm, 3, sq, 500, 4, 2, d, softcap=cap, starts=ints(3, 64, 300 - sq), window=50)
    check(lm, 3, sq, 500, 4, 2, d, softcap=cap, starts=ints(3, 64, 290 - sq), window=50, causal=False)
    check(lm, 3, sq, 500, 4, 2, d, softcap=cap, starts=ints(0, 131, 499 - sq), prefix=ints(150, 10, 0))


@pytest.mark.parametrize("sq,sk", [(1, 3000), (3, 3000), (64, 2500)])
def test_long_caches_past_their_last_position(lm, sq, sk):
    check(lm, 2, sq, sk, 4, 1, 64, starts=ints(0, sk - sq - 70))


@pytest.mark.parametrize("d,cap", [(64, 0.0), (128, 0.0), (128, 20.0), (80, 0.0)])
def test_queries_that_see_nothing(lm, d, cap):
    check(lm, 1, 130, 40, 4, 2, d, softcap=cap)                                         # more queries than keys
    check(lm, 2, 200, 200, 4, 2, d, softcap=cap, starts=ints(-70, 60))
    check(lm, 2, 200, 200, 4, 2, d, softcap=cap, starts=ints(-70, 60), window=30)
    check(lm, 2, 200, 200, 4, 2, d, softcap=cap, starts=ints(-130, 150), window=30, causal=False)
    check(lm, 2, 200, 200, 4, 2, d, softcap=cap, starts=ints(-200, 400), window=30)     # nobody sees anything
    check(lm, 2, 200, 200, 4, 2, d, softcap=cap, starts=ints(-70, 20), lengths=ints(130, 0))
    check(lm, 2, 200, 200, 4, 2, d, softcap=cap, starts=ints(-70, 20), prefix=ints(0, 9), keys=False)
