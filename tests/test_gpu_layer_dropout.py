"""Dropout against its definition: the same elements dropped, the others exact."""

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


def want(x, p, seed, offset=0):
    f = ref.factors(x.numel(), p, seed, offset).view(x.shape)
    # float32 arithmetic, rounded once; a dropped element is +0 whatever x holds
    y = (x.float().cpu() * f.float()).to(x.dtype)
    return torch.where(f == 0, torch.zeros_like(y), y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2049, 5000])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_against_the_definition(lm, dtype, n, p):
    x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dtype).cuda()
    seed, offset = 0x123456789ABCDEF0, (1 << 32) - 3
    got = lm.dropout(x, p, seed, offset)
    assert got.dtype is dtype and torch.equal(got.cpu(), want(x, p, seed, offset))
