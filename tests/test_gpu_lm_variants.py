"""Variants and loops of the language-model kernels that only some sizes reach:
gradients of every extra at padded head sizes, walks of more than 64 tiles,
joins of more than 64 chunks, and sorts whose lists overflow."""

import math

import pytest
import torch

from . import lm_bounds
from . import lm_reference as ref
from .test_gpu_lm_attention import MASKS, check, docs, ints, make, masks
from .test_gpu_lm_other import check_embed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm as m
    return m


@pytest.mark.parametrize("name", MASKS)
@pytest.mark.parametrize("d", [72, 80, 96, 104, 120])
def test_masks_at_padded_head_sizes(lm, name, d):
    """200 keys: the second block of 128 is a partial one."""
    b, s, hq, hkv = 2, 200, 4, 2
    check(lm, *make(b, s, s, hq, hkv, d), **masks(MASKS[name], b, s, s, hq))


@pytest.mark.parametrize("s", [97, 129, 161, 255])
@pytest.mark.parametrize("d", [80, 112, 128])
def test_partial_blocks_of_keys(lm, s, d):
    """Waves (and pairs of them) whose 32 keys end early, with every extra."""
    slopes = torch.tensor([0.5, 0.1, 0.02]).cuda()
    for kw in (dict(softcap=20.0), dict(softcap=20.0, slopes=slopes, causal=False), dict(slopes=slopes, window=60)):
        check(lm, *make(1, s, s, 3, 1, d, seed=s), **kw)


def long_check(lm, s, d, softcap=0.0, **mask):
    """4500 queries over 4500 keys: 71 tiles either way; the masks vectorised."""
    print(f"attention of {s} tokens, heads of {d}, cap {softcap} {sorted(mask)}", flush=True)
    q, k, v, dout = make(1, s, s, 2, 1, d)
    i, j = torch.arange(s)[:, None], torch.arange(s)[None]
    vis = (j <= i) if mask.get("causal", True) else torch.ones(s, s, dtype=torch.bool)
    if mask.get("window"):
        vis &= (i - j).abs() < mask["window"]
    if "prefix" in mask:
        vis |= j < int(mask["prefix"][0])
    if "documents" in mask:
        vis &= mask["documents"].cpu()[0][:, None] == mask["documents"].cpu()[0][None]
    want, tol = lm_bounds.attention(q, k, v, dout, vis[None], torch.arange(s)[None], softcap=softcap)
    out, lse = lm.attention(q, k, v, softcap=softcap, **mask)
    grads = lm.attention_backward(dout, q, k, v, out, lse, softcap=softcap, **mask)
    torch.cuda.synchronize()
    for t, name in zip((out, lse, *grads), ("out", "lse", "dq", "dk", "dv")):
        ref.close(t, want[name], tol[name], name)


@pytest.mark.parametrize("d,cap", [(64, 0.0), (128, 100.0)])
@pytest.mark.parametrize("mask", ["causal", "everything", "window", "documents", "few documents", "prefix"])
def test_walks_of_more_than_64_tiles(lm, d, cap, mask):
    s = 4500
    kw = {"causal": {}, "everything": dict(causal=False), "window": dict(window=700),
          "documents": dict(documents=docs(1, s, 900)),
          # the same number again far on: only the first and the last tiles of a walk hold keys
          "few documents": dict(documents=((torch.arange(s) // 64 + 1) % 70).int()[None].cuda(), causal=False),
          "prefix": dict(prefix=ints(130), window=40)}[mask]
    long_check(lm, s, d, softcap=cap, **kw)


@pytest.mark.parametrize("hq,hkv,d,kw", [(2, 1, 64, {}), (1, 1, 128, dict(softcap=30.0)), (8, 1, 96, dict(window=69000))])
def test_more_than_64_chunks_of_keys(lm, hq, hkv, d, kw):
    check(lm, *make(1, 1, 70001, hq, hkv, d), backward=False, **kw)


@pytest.mark.parametrize("b,sq,hq,hkv,d", [(3, 5, 16, 2, 64), (20, 2, 32, 1, 128), (2, 9, 24, 6, 80)])
def test_a_few_queries_of_many_heads(lm, b, sq, hq, hkv, d):
    """More than 32 rows (query, head) for each key head."""
    check(lm, *make(b, sq, 700, hq, hkv, d))


@pytest.mark.parametrize("n,vocab", [(60000, 50257), (40000, 3), (70000, 700)])
def test_sorts_whose_lists_overflow(lm, n, vocab):
    """A third of the tokens are one token (padding): more than 1024 entries of
    one workgroup's rows in a sixteenth of the tokens."""
    g = torch.Generator().manual_seed(n)
    tokens = (torch.rand(n, generator=g, dtype=torch.float64) ** 4 * vocab).long()
    tokens[torch.rand(n, generator=g) < 0.34] = vocab - 1
    check_embed(lm, tokens.cuda(), vocab, 24, torch.float32, torch.bfloat16, math.sqrt(24))
    check_embed(lm, tokens.int().cuda(), vocab, 17, torch.bfloat16, torch.float32, 1.0)
    tokens[n // 2:] = vocab - 1  # whole parts of one token
    check_embed(lm, tokens.cuda(), vocab, 8, torch.float32, torch.float32, 1.0)
