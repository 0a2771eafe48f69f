"""The operators together: the example decoder trains, and its generation over
a cache agrees with its whole forward pass."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from newton_schulz_09_amd import lm_example as m
    return m


def test_training_lowers_the_loss(example):
    def run():
        model = example.Decoder(vocab=128, seed=3)
        start = torch.arange(4, device="cuda")[:, None]
        tokens = (start * 7 + torch.arange(130, device="cuda")) % 97
        documents = (torch.arange(130, device="cuda") // 50).int().expand(4, 130).contiguous()
        return model, [model.step(tokens, documents).item() for _ in range(30)]

    model, losses = run()
    assert losses[-1] < 0.5 * losses[0], losses
    assert all(torch.isfinite(m).all() for m in model.matrices + model.vectors)


def test_generation_agrees_with_the_whole_pass(example):
    model = example.Decoder(vocab=128, layers=2, seed=5)
    g = torch.Generator().manual_seed(0)
    prompt = torch.randint(0, 128, (3, 21), generator=g).cuda()
    lengths = torch.tensor([21, 1, 9]).cuda()
    tokens, logits = model.generate(prompt, lengths, 6)
    for i, n in enumerate(lengths.tolist()):
        whole = torch.cat([prompt[i, :n], tokens[i, :-1]])[None]
        with torch.no_grad():
            want = model.logits(whole)[n - 1:]
        # both sides round activations to bfloat16 at the same places, and
        # sums in another order move some by a step (2^-7 of the value at
        # most): the residual stream is rounded 3 times in 2 layers, heads and
        # projections 4 times a layer, so about a dozen steps of the norm of x
        # against a unit-variance table
        x = want.double()
        off = (logits[i].double() - x).norm() / x.norm()
        assert off < 12 * 2.0 ** -8, (i, off)
        assert torch.equal(logits[i].argmax(-1), tokens[i])


def test_the_examples_main(example, capsys):
    example.main()
    assert "continuations" in capsys.readouterr().out
