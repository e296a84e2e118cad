"""Two state space blocks built from the package's operators, trained for a few
steps and then served: a prompt batch with sequences of different lengths, and
single tokens that continue from its states.

* HeadBlock: projection, short convolution, the scan with one decay per head
  (ssd), gated norm, projection.
* ChannelBlock: projection, short convolution, the selective scan (a decay per
  channel and state) with its gate, projection.

    python examples/blocks.py [--steps N]

Everything between the projections runs in the package's kernels.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba_ssd_forward_gb300 as ssd  # noqa: E402

IO = torch.bfloat16


class Block:
    """Parameters by name: projections in bf16, the small ones in fp32."""

    def __init__(self):
        self.p = {}

    def add(self, name, value):
        self.p[name] = value.cuda().requires_grad_()

    def linear(self, name, rows, cols):
        self.add(name, (torch.randn(rows, cols) / math.sqrt(cols)).to(IO))


def _steps_bias(n):
    """softplus^-1 of steps spread over 1e-3 .. 1e-1."""
    s = torch.exp(math.log(1e-3) + torch.rand(n) * math.log(100.0))
    return s + torch.log(-torch.expm1(-s))


class HeadBlock(Block):
    def __init__(self, width=128, heads=4, dstate=64, conv=4):
        super().__init__()
        self.heads, self.inner, self.dstate = heads, 64 * heads, dstate
        d, s = self.inner, dstate
        self.linear("w_in", 2 * d + 2 * s + heads, width)
        self.add("conv", torch.randn(d + 2 * s, conv) * conv ** -0.5)
        self.add("conv_bias", torch.zeros(d + 2 * s))
        self.add("A_log", torch.log(1.0 + torch.arange(heads).float()))
        self.add("D", torch.ones(heads))
        self.add("dt_bias", _steps_bias(heads))
        self.add("norm", torch.ones(d))
        self.linear("w_out", width, d)

    def _split(self, x):
        d, s = self.inner, self.dstate
        return torch.split(F.linear(x, self.p["w_in"]), [d, d + 2 * s, self.heads], dim=-1)

    def _parts(self, xbc):
        """x, B and C of the convolved channels, dense as the scan takes them."""
        b, L = xbc.shape[:2]
        x, B, C = torch.split(xbc, [self.inner, self.dstate, self.dstate], dim=-1)
        return (x.reshape(b, L, self.heads, 64), B.reshape(b, L, 1, -1), C.reshape(b, L, 1, -1))

    def _decay(self):
        return -torch.exp(self.p["A_log"])

    def train_forward(self, x):
        p = self.p
        z, xbc, dt = self._split(x)
        xbc, _ = ssd.causal_conv(xbc, p["conv"], p["conv_bias"])
        u, B, C = self._parts(xbc)
        dt = F.softplus(dt.float() + p["dt_bias"]).to(IO)
        y, _ = ssd.ssd(u.contiguous(), dt.contiguous(), self._decay(), B.contiguous(),
                       C.contiguous(), p["D"], chunk=64)
        y = ssd.gated_norm(y.flatten(2), p["norm"], z=z)
        return F.linear(y, p["w_out"])

    @torch.no_grad()
    def prompt(self, x, lengths):
        """Outputs of padded prompts, and the states after each one's end."""
        p, L = self.p, x.shape[1]
        z, xbc, dt = self._split(x)
        xbc, conv_state = ssd.causal_conv_forward(xbc, p["conv"], p["conv_bias"], lengths=lengths)
        u, B, C = self._parts(xbc)
        # a step of zero leaves the state alone: the padding changes nothing
        real = torch.arange(L, device=x.device)[None, :, None] < lengths[:, None, None]
        dt = torch.where(real, F.softplus(dt.float() + p["dt_bias"]), 0.0).to(IO)
        y, state = ssd.forward(u.contiguous(), dt, self._decay(), B.contiguous(), C.contiguous(),
                               p["D"], chunk=64)
        y = ssd.gated_norm_forward(y.flatten(2), p["norm"], z=z)
        return F.linear(y, p["w_out"]), (conv_state, state)

    @torch.no_grad()
    def token(self, x, states):
        """One token of every sequence, x [b, width]; the states move on."""
        p, (conv_state, state) = self.p, states
        z, xbc, dt = self._split(x)
        xbc = ssd.causal_conv_step(xbc, p["conv"], p["conv_bias"], conv_state)
        u, B, C = (t[:, 0].contiguous() for t in self._parts(xbc[:, None]))
        dt = F.softplus(dt.float() + p["dt_bias"]).to(IO)
        y = ssd.decode_step(u, dt, self._decay(), B, C, p["D"], state)
        return F.linear(ssd.gated_norm_forward(y.flatten(1), p["norm"], z=z), p["w_out"])


class ChannelBlock(Block):
    def __init__(self, width=128, inner=256, dstate=16, rank=8, conv=4):
        super().__init__()
        self.inner, self.dstate, self.rank = inner, dstate, rank
        self.linear("w_in", 2 * inner, width)
        self.add("conv", torch.randn(inner, conv) * conv ** -0.5)
        self.add("conv_bias", torch.zeros(inner))
        self.linear("w_x", rank + 2 * dstate, inner)
        self.linear("w_dt", inner, rank)
        self.add("dt_bias", _steps_bias(inner))
        self.add("A_log", torch.log(1.0 + torch.arange(dstate).float()).repeat(inner, 1))
        self.add("D", torch.ones(inner))
        self.linear("w_out", width, inner)

    def _scan_inputs(self, u, z):
        """The scan's arguments from the convolved channels, any leading axes."""
        p, n = self.p, self.dstate
        r, B, C = torch.split(F.linear(u, p["w_x"]), [self.rank, n, n], dim=-1)
        return (u, F.linear(r, p["w_dt"]), -torch.exp(p["A_log"]), B.unflatten(-1, (1, n)),
                C.unflatten(-1, (1, n)), p["D"], z, p["dt_bias"])

    def train_forward(self, x):
        p = self.p
        u, z = F.linear(x, p["w_in"]).chunk(2, dim=-1)
        u, _ = ssd.causal_conv(u, p["conv"], p["conv_bias"])
        y, _ = ssd.selective_scan(*self._scan_inputs(u, z), dt_softplus=True)
        return F.linear(y, p["w_out"])

    @torch.no_grad()
    def prompt(self, x, lengths):
        p = self.p
        u, z = F.linear(x, p["w_in"]).chunk(2, dim=-1)
        u, conv_state = ssd.causal_conv_forward(u, p["conv"], p["conv_bias"], lengths=lengths)
        y, state = ssd.selective_scan_forward(*self._scan_inputs(u, z), lengths=lengths,
                                              dt_softplus=True)
        return F.linear(y, p["w_out"]), (conv_state, state)

    @torch.no_grad()
    def token(self, x, states):
        p, (conv_state, state) = self.p, states
        u, z = F.linear(x, p["w_in"]).chunk(2, dim=-1)
        u = ssd.causal_conv_step(u, p["conv"], p["conv_bias"], conv_state)
        y = ssd.selective_scan_step(*self._scan_inputs(u, z), state, dt_softplus=True)
        return F.linear(y, p["w_out"])


def train(block, steps=8, batch=4, tokens=96, width=128, rate=0.1, max_norm=1.0, seed=0):
    """Fits a random target by clipped gradient descent; the losses."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(batch, tokens, width, generator=g, device="cuda").to(IO)
    target = torch.randn(batch, tokens, width, generator=g, device="cuda")
    losses = []
    for _ in range(steps):
        loss = F.mse_loss(block.train_forward(x).float(), target)
        losses.append(float(loss.detach()))
        params = list(block.p.values())
        grads = [t.contiguous() for t in torch.autograd.grad(loss, params)]
        ssd.clip_grad_norm(grads, max_norm)
        with torch.no_grad():
            for p, d in zip(params, grads):
                p -= rate * d
    return losses


def serve(block, lengths=(40, 1, 23), new=5, width=128, seed=1):
    """Largest difference between tokens served one by one after a padded prompt
    and the same sequences run whole, relative to the outputs' size."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    total = max(lengths) + new
    x = torch.randn(len(lengths), total, width, generator=g, device="cuda").to(IO)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    _, states = block.prompt(x[:, :max(lengths)], n)
    rows = torch.arange(len(lengths), device="cuda")
    served = torch.stack([block.token(x[rows, n.long() + k], states) for k in range(new)], 1)
    whole, _ = block.prompt(x, n + new)
    at = n.long()[:, None] + torch.arange(new, device="cuda")
    ref = whole[rows[:, None], at].float()
    return float((served.float() - ref).norm() / ref.norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    torch.manual_seed(0)
    for block in (HeadBlock(), ChannelBlock()):
        losses = train(block, steps=args.steps)
        off = serve(block)
        print(f"{type(block).__name__}: loss {losses[0]:.4f} -> {losses[-1]:.4f} in "
              f"{args.steps} steps; served tokens within {off:.1e} of the whole sequences")


if __name__ == "__main__":
    main()
