"""A small decoder trained and sampled with this package's operators: scaled
embedding, norm and rotation of query and key heads, attention over packed
documents, their gradients, and Muon steps on the matrices.

    python -m newton_schulz_09_amd.lm_example

``Embedding``, ``NormRotation`` and ``Attention`` show how the operators of
``lm`` join torch's autograd; ``Decoder.generate`` runs the same operators on
single tokens over a cache.
"""

import math

import torch

from . import lm, muon


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale):
        ctx.save_for_backward(tokens)
        ctx.scale, ctx.vocab, ctx.dtype = scale, table.shape[0], table.dtype
        return lm.embedding(tokens, table, scale=scale, dtype=torch.bfloat16)

    @staticmethod
    def backward(ctx, dout):
        tokens, = ctx.saved_tensors
        return None, lm.embedding_backward(dout.contiguous(), tokens, ctx.vocab, scale=ctx.scale, dtype=ctx.dtype), None


class NormRotation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, q_weight, k_weight):
        ctx.save_for_backward(q, k, table, positions, q_weight, k_weight)
        return lm.qk_norm_rope(q, k, table, positions=positions, q_weight=q_weight, k_weight=k_weight)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, table, positions, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dqw, dkw = lm.qk_norm_rope_backward(dq, dk, q, k, table, positions=positions, q_weight=q_weight,
                                                    k_weight=k_weight)
        return dq, dk, None, None, dqw, dkw


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, documents, softcap):
        out, lse = lm.attention(q, k, v, documents=documents, softcap=softcap)
        ctx.save_for_backward(q, k, v, out, lse, documents)
        ctx.softcap = softcap
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, documents = ctx.saved_tensors
        dq, dk, dv = lm.attention_backward(dout.contiguous(), q, k, v, out, lse, documents=documents,
                                           softcap=ctx.softcap)
        return dq, dk, dv, None, None


class Decoder:
    """Layers of attention alone, with residuals; logits against the embedding's table."""

    def __init__(self, vocab=512, layers=2, heads=4, kv_heads=2, d=64, limit=1024, softcap=30.0, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.d, self.softcap, self.device = heads, kv_heads, d, softcap, torch.device(device)
        self.width = width = heads * d
        self.scale = math.sqrt(width)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).requires_grad_()

        self.table = normal(vocab, width, std=1.0 / self.scale)
        self.layers = [{"qkv": normal(width, (heads + 2 * kv_heads) * d, std=width ** -0.5),
                        "out": normal(width, width, std=0.5 * width ** -0.5),
                        "qw": torch.ones(d, device=device, requires_grad=True),
                        "kw": torch.ones(d, device=device, requires_grad=True)} for _ in range(layers)]
        freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=device) / d)
        angle = torch.arange(limit, dtype=torch.float64, device=device)[:, None] * freq
        self.angles = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        # the matrices, which Muon updates, and its state
        self.matrices = [m for layer in self.layers for m in (layer["qkv"], layer["out"])]
        self.buffers = [torch.zeros_like(m) for m in self.matrices]
        self.vectors = [v for layer in self.layers for v in (layer["qw"], layer["kw"])]

    def _heads(self, x, layer, positions):
        """Rotated queries and keys, and values, of x (batch, s, width)."""
        b, s, _ = x.shape
        unit = x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)
        qkv = (unit.bfloat16().reshape(b * s, -1) @ layer["qkv"].bfloat16()).view(b, s, -1, self.d)
        h, u = self.heads, self.kv_heads
        q, k = NormRotation.apply(qkv[:, :, :h], qkv[:, :, h:h + u], self.angles, positions, layer["qw"], layer["kw"])
        return q, k, qkv[:, :, h + u:]

    def _after(self, x, heads, layer):
        b, s, _ = x.shape
        return x + (heads.reshape(b * s, -1) @ layer["out"].bfloat16()).view(b, s, -1)

    def _logits(self, x):
        return x.float().reshape(-1, self.width) @ self.table.t()

    def logits(self, tokens, documents=None):
        """(batch * s, vocab) logits of tokens (batch, s)."""
        b, s = tokens.shape
        positions = torch.arange(s, dtype=torch.int32, device=self.device).expand(b, s).contiguous()
        x = Embedding.apply(tokens, self.table, self.scale)
        for layer in self.layers:
            q, k, v = self._heads(x, layer, positions)
            x = self._after(x, Attention.apply(q, k, v, documents, self.softcap), layer)
        return self._logits(x)

    def step(self, tokens, documents=None, lr=0.02, lr_rest=0.5):
        """One training step on the next tokens; returns the loss (a tensor)."""
        logits = self.logits(tokens[:, :-1].contiguous(), None if documents is None else documents[:, :-1].contiguous())
        loss = torch.nn.functional.cross_entropy(logits, tokens[:, 1:].reshape(-1))
        rest = [self.table, *self.vectors]
        grads = torch.autograd.grad(loss, self.matrices + rest)
        n = len(self.matrices)
        with torch.no_grad():
            muon.ns5_batched([g.contiguous() for g in grads[:n]], [m.detach() for m in self.matrices],
                             bufs=self.buffers, mu=0.95, lr=lr)
            for p, g in zip(rest, grads[n:]):
                p -= lr_rest * g
        return loss.detach()

    @torch.no_grad()
    def generate(self, prompt, lengths, count):
        """Greedy continuations of prompts (batch, s), whose first lengths[i]
        tokens count: (batch, count) tokens, and the logits each came from."""
        b, s = prompt.shape
        lengths = lengths.to(torch.int32)
        cache = [torch.zeros(2, b, s + count, self.kv_heads, self.d, dtype=torch.bfloat16, device=self.device)
                 for _ in self.layers]
        rows = torch.arange(b, device=self.device)
        # the prompts
        positions = torch.arange(s, dtype=torch.int32, device=self.device).expand(b, s).contiguous()
        zero = torch.zeros_like(lengths)
        x = lm.embedding(prompt, self.table, scale=self.scale, dtype=torch.bfloat16)
        for layer, (ck, cv) in zip(self.layers, cache):
            q, k, v = self._heads(x, layer, positions)
            ck[:, :s], cv[:, :s] = k, v
            out, _ = lm.attention(q, k, v, softcap=self.softcap, lengths=lengths, starts=zero)
            x = self._after(x, out, layer)
        x = x[rows, lengths.long() - 1][:, None]
        tokens, every = [], []
        for i in range(count):
            logits = self._logits(x)
            every.append(logits)
            tokens.append(logits.argmax(-1))
            if i + 1 == count:
                break
            # one token a sequence, at position lengths[i]
            x = lm.embedding(tokens[-1][:, None], self.table, scale=self.scale, dtype=torch.bfloat16)
            after = lengths + 1
            for layer, (ck, cv) in zip(self.layers, cache):
                q, k, v = self._heads(x, layer, lengths[:, None].contiguous())
                ck[rows, lengths.long()], cv[rows, lengths.long()] = k[:, 0], v[:, 0]
                out, _ = lm.attention(q, ck, cv, softcap=self.softcap, lengths=after, starts=lengths)
                x = self._after(x, out, layer)
            lengths = after
        return torch.stack(tokens, 1), torch.stack(every, 1)


def main():
    model = Decoder()
    # counting sequences, two documents to a row
    start = torch.arange(8, device="cuda")[:, None]
    half = torch.arange(128, device="cuda")[None]
    tokens = torch.cat([(start * 7 + half) % 97, (start * 5 + 3 * half) % 97], 1)
    documents = torch.cat([torch.zeros_like(half), torch.ones_like(half)], 1).expand(8, 256).int().contiguous()
    for i in range(60):
        loss = model.step(tokens, documents)
        if i % 10 == 0 or i == 59:
            print(f"step {i}: loss {loss.item():.4f}")
    out, _ = model.generate(tokens[:2, :20].contiguous(), torch.tensor([20, 12], device="cuda"), 8)
    print("continuations:", out.tolist())


if __name__ == "__main__":
    main()
