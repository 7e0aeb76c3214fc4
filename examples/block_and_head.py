"""The end of a language model in training and in decoding: a gated feed-forward block with its
residual, the vocabulary head's cross-entropy, clipped gradients.

    python examples/block_and_head.py [--tokens N] [--width d] [--ffn F] [--vocab V] [--steps K]
                                      [--dtype bf16|f32]

Training step: h = gated_linear(x, Wg, Wu), y = linear_act(h, Wd, bias, residual=x), loss =
linear_cross_entropy(y, W, labels), backward, clip_grad_norm_, SGD.  Neither the block's
pre-activations nor the N x V logits exist in memory at any time.  Decoding: the same block and the
head as a product for one token at a time.  Data is synthetic: each token's label is a fixed
function of its (fixed) embedding, so the loss falls.

    python examples/block_and_head.py --from-tokens ...

The same from tokens to tokens: embedding (its table is the head's too), layer_norm, the block,
layer_norm, the head's loss, with the table's two gradients added by autograd; then the next tokens by
sample_tokens, one after the other (each depends on the one before alone).
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import memory_bounded_linear_gb300 as lce  # noqa: E402


class FeedForward(torch.nn.Module):
    """y = act(x Wg^T) * (x Wu^T) Wd^T + bias + x."""

    def __init__(self, width, ffn, activation="silu", device=None, dtype=None):
        super().__init__()
        kw = dict(device=device, dtype=dtype)
        self.activation = activation
        self.gate = torch.nn.Parameter(torch.randn(ffn, width, **kw) * width ** -0.5)
        self.up = torch.nn.Parameter(torch.randn(ffn, width, **kw) * width ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(width, ffn, **kw) * ffn ** -0.5)
        self.bias = torch.nn.Parameter(torch.zeros(width, **kw))

    def forward(self, x):
        h = lce.gated_linear(x, self.gate, self.up, self.activation)
        return lce.linear_act(h, self.down, self.bias, residual=x)


class BlockAndHead(torch.nn.Module):
    def __init__(self, width, ffn, vocab, device=None, dtype=None):
        super().__init__()
        self.block = FeedForward(width, ffn, device=device, dtype=dtype)
        self.head = torch.nn.Parameter(
            torch.randn(vocab, width, device=device, dtype=dtype) * width ** -0.5)

    def loss(self, x, labels):
        return lce.linear_cross_entropy(self.block(x).contiguous(), self.head, labels)

    @torch.no_grad()
    def next_token(self, x):
        """The most likely token after each of a few positions x [n, width]."""
        return lce.linear_act(self.block(x), self.head).argmax(-1)


class TokenModel(torch.nn.Module):
    """Tokens in, tokens out: h = LN2(block(LN1(s E[t]))), logits h E^T."""

    def __init__(self, width, ffn, vocab, device=None, dtype=None):
        super().__init__()
        kw = dict(device=device, dtype=dtype)
        self.scale = width ** 0.5
        self.table = torch.nn.Parameter(torch.randn(vocab, width, **kw) * width ** -0.5)
        self.norm1, self.norm2 = (torch.nn.ParameterList([torch.nn.Parameter(torch.ones(width, **kw)),
                                                          torch.nn.Parameter(torch.zeros(width, **kw))])
                                  for _ in range(2))
        self.block = FeedForward(width, ffn, **kw)

    def hidden(self, tokens):
        """tokens [...] -> h [..., width]; padding (-100) has an embedding of zeros."""
        x = lce.layer_norm(lce.embedding(tokens, self.table, self.scale), *self.norm1)
        return lce.layer_norm(self.block(x), *self.norm2)

    def loss(self, tokens, labels):
        h = self.hidden(tokens)
        return lce.linear_cross_entropy(h.reshape(-1, h.shape[-1]), self.table, labels.reshape(-1))

    @torch.no_grad()
    def head(self):
        """The table as linear_act's weight, whose rows come in eights: behind an odd vocabulary's there are zeros."""
        more = -self.table.shape[0] % 8
        return torch.nn.functional.pad(self.table, (0, 0, 0, more)) if more else self.table

    @torch.no_grad()
    def logits(self, tokens, head=None):
        """Logits after each of tokens [n]; ``head`` is self.head(), where there is one already."""
        head = self.head() if head is None else head
        return lce.linear_act(self.hidden(tokens), head)[..., :self.table.shape[0]]

    @torch.no_grad()
    def next_tokens(self, tokens, head=None, **sampling):
        """A token after each of tokens [n]."""
        return lce.sample_tokens(self.logits(tokens, head), **sampling)

    @torch.no_grad()
    def generate(self, tokens, steps, **sampling):
        out, head = [tokens], self.head()
        for _ in range(steps):
            out.append(self.next_tokens(out[-1], head, **sampling))
        return torch.stack(out, -1)


def train(model, x, labels, steps, lr=2.0, max_norm=1.0):
    """Plain SGD on one batch; returns the losses and the gradient norms before clipping, read back
    once at the end."""
    losses, norms = [], []
    for _ in range(steps):
        model.zero_grad(set_to_none=True)
        loss = model.loss(x, labels)
        loss.backward()
        norms.append(lce.clip_grad_norm_(model.parameters(), max_norm))
        losses.append(loss.detach())
        with torch.no_grad():
            for p in model.parameters():
                p.add_(p.grad, alpha=-lr)
    return torch.stack(losses).tolist(), torch.stack(norms).tolist()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=1000)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--ffn", type=int, default=2048)
    p.add_argument("--vocab", type=int, default=4096)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    p.add_argument("--from-tokens", action="store_true")
    a = p.parse_args(argv)
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[a.dtype]
    torch.manual_seed(0)
    if a.from_tokens:
        model = TokenModel(a.width, a.ffn, a.vocab, device="cuda", dtype=dtype)
        tokens = torch.randint(0, a.vocab, (a.tokens,), device="cuda")
        losses, norms = train(model, tokens, (tokens * 7 + 3) % a.vocab, a.steps, lr=0.5)
        print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps; "
              f"gradient norm {norms[0]:.3f} -> {norms[-1]:.3f}")
        text = model.generate(tokens[:4], 8, temperature=0.8, top_k=50, top_p=0.95)
        print("tokens", text.tolist())
        return losses, norms, text
    model = BlockAndHead(a.width, a.ffn, a.vocab, device="cuda", dtype=dtype)
    x = torch.randn(a.tokens, a.width, device="cuda").to(dtype)
    labels = torch.randint(0, a.vocab, (a.tokens,), device="cuda")
    losses, norms = train(model, x, labels, a.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps; "
          f"gradient norm {norms[0]:.3f} -> {norms[-1]:.3f}")
    # decoding: one position at a time gives what the batch gives
    few = x[:8]
    together = model.next_token(few)
    one_by_one = torch.cat([model.next_token(few[i:i + 1]) for i in range(few.shape[0])])
    print("tokens", together.tolist(), "one by one", one_by_one.tolist())
    return losses, norms, together, one_by_one


if __name__ == "__main__":
    main()
