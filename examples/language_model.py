"""A small language model of the two blocks of blocks.py, with the package's operators
around them: the residual's addition and the norm in front of each block, the loss over
the vocabulary without its logits, clipped gradients, and orthogonalised updates of the
matrices.

    python examples/language_model.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import mamba_ssd_forward_gb300 as ssd  # noqa: E402
from blocks import IO, ChannelBlock, HeadBlock  # noqa: E402


class Model:
    """Embedding (which is the vocabulary's matrix too), two blocks, a norm in front of
    each and of the loss.  The residual stream is fp32."""

    def __init__(self, words=512, width=128):
        self.width = width
        self.blocks = [HeadBlock(width), ChannelBlock(width)]
        self.p = {"words": (torch.randn(words, width) * width ** -0.5).to(IO).cuda()
                  .requires_grad_()}
        for i, b in enumerate(self.blocks):
            self.p[f"norm{i}"] = torch.ones(width, device="cuda", requires_grad=True)
            self.p |= {f"{i}.{k}": v for k, v in b.p.items()}
        self.p["norm"] = torch.ones(width, device="cuda", requires_grad=True)

    def _embed(self, tokens):
        return self.p["words"][tokens.clamp(min=0)]

    def _stream(self, x):
        return torch.zeros(x.shape, dtype=torch.float32, device=x.device)

    def hidden(self, tokens, norm=ssd.add_norm):
        x = self._embed(tokens)
        stream = self._stream(x)
        for i, b in enumerate(self.blocks):
            y, stream = norm(x, stream, self.p[f"norm{i}"])
            x = b.train_forward(y)
        return norm(x, stream, self.p["norm"])[0]

    def loss(self, tokens, norm=ssd.add_norm, entropy=ssd.linear_cross_entropy):
        """The mean loss of each token's successor; -100 stands for none."""
        x = self.hidden(tokens[:, :-1], norm)
        return entropy(x, self.p["words"], tokens[:, 1:].contiguous(), reduction="mean")

    @torch.no_grad()
    def prompt(self, tokens):
        """The next word after each prompt, and the blocks' states."""
        lengths = torch.full((len(tokens),), tokens.shape[1], dtype=torch.int32, device="cuda")
        x, states = self._embed(tokens), []
        stream = self._stream(x)
        for i, b in enumerate(self.blocks):
            y, stream = ssd.add_norm_forward(x, stream, self.p[f"norm{i}"], total=stream)
            x, s = b.prompt(y, lengths)
            states.append(s)
        return self._word(x[:, -1], stream[:, -1]), states

    @torch.no_grad()
    def token(self, words, states):
        x = self._embed(words)
        stream = self._stream(x)
        for i, b in enumerate(self.blocks):
            y, stream = ssd.add_norm_forward(x, stream, self.p[f"norm{i}"], total=stream)
            x = b.token(y, states[i])
        return self._word(x, stream)

    def _word(self, x, stream):
        y, _ = ssd.add_norm_forward(x.contiguous(), stream.contiguous(), self.p["norm"])
        return (y @ self.p["words"].t()).argmax(-1)


def train(model, tokens, steps=8, rate=0.02, max_norm=1.0):
    """Clipped gradients; matrices move along their orthogonalised update."""
    losses = []
    params = list(model.p.values())
    for _ in range(steps):
        loss = model.loss(tokens)
        losses.append(float(loss.detach()))
        grads = [g.contiguous() for g in torch.autograd.grad(loss, params)]
        ssd.clip_grad_norm(grads, max_norm)
        with torch.no_grad():
            for (name, p), g in zip(model.p.items(), grads):
                if p.dim() == 2 and p.dtype == IO and name != "words":
                    m, n = p.shape
                    g = ssd.orthogonalize(g) * max(1.0, m / n) ** 0.5
                p -= rate * g.to(p.dtype)
    return losses


def serve(model, tokens, new=4):
    """`new` words after each prompt, the likeliest each time: [b, new]."""
    word, states = model.prompt(tokens)
    out = [word]
    for _ in range(new - 1):
        out.append(model.token(out[-1], states))
    return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Model()
    tokens = torch.randint(0, 512, (4, 129), device="cuda")
    losses = train(model, tokens, args.steps)
    words = serve(model, tokens[:, :32])
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {args.steps} steps; then served "
          f"{words.shape[1]} words after each of {words.shape[0]} prompts")


if __name__ == "__main__":
    main()
