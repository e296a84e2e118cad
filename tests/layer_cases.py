"""Seeded inputs and tolerances shared by the GPU tests of the operators
around the scan.

Tolerances are relative L2 over a tensor, fixed from the arithmetic:
  U = 2^-24 the fp32 rounding.  An elementwise result of a few fp32 operations
  with one fast exponential and a division (2 to 3 ulp each, and |v| U for an
  exponent of size |v| <= 20) is within 32 U ~ 2e-6; E = 5e-6.
  A sum of n terms of either sign adds sqrt(n) U of its own size while the
  terms' sizes add up to sqrt(n) times the sum: n U for it, capped by E for
  short ones.
  A recurrence over L tokens multiplies L decays, each off by up to 4 U: 4 L U
  on top.
  A bf16 output is rounded once to 8 significant bits: at most 2^-8 of every
  element, so 2^-8 of the norm.
"""
import numpy as np
import torch

U = 2.0 ** -24
E = 5e-6
BF16 = 2.0 ** -8

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def tol(dtype, tokens=0, terms=0):
    return E + 4 * tokens * U + terms * U + (BF16 if dtype == torch.bfloat16 else 0.0)


def to64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, limit, what):
    got, ref = to64(got), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    norm = np.linalg.norm(ref)
    off = np.linalg.norm(got - ref)
    assert off <= limit * norm + 1e-30, f"{what}: off by {off / max(norm, 1e-300):.3e}, limit {limit:.3e}"


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cpu")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0, wide=0, device="cuda"):
        """N(0, scale^2); with `wide`, the last columns of rows that are wider."""
        t = torch.randn(*shape[:-1], shape[-1] + wide, generator=self.g) * scale
        return t.to(dtype).to(device)[..., wide:]

    def uniform(self, *shape, device="cuda"):
        return torch.rand(*shape, generator=self.g).to(device)


def lengths_of(n):
    return None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")


def conv_inputs(b, L, D, W, dtype, seed=0, wide=0, state=True, bias=True):
    r, io = Draw(seed), DTYPES[dtype]
    return dict(x=r.normal(b, L, D, dtype=io, wide=wide), weight=r.normal(D, W, scale=0.5),
                bias=r.normal(D, scale=0.3) if bias else None,
                state=r.normal(b, W - 1, D, dtype=io) if state else None), \
        r.normal(b, L, D, dtype=io, wide=wide), r.normal(b, W - 1, D, dtype=io)


def scan_inputs(b, L, D, N, G, dtype, seed=0, wide=0, h0=True, z=True, skip=True, bias=True):
    """Steps of about 1e-3 to 1e-1 with softplus (the bias at -4), decays of
    -1 to -N."""
    r, io = Draw(seed), DTYPES[dtype]
    bc = r.normal(b, L, 2 * G * N, dtype=io, wide=wide)
    s = dict(u=r.normal(b, L, D, dtype=io), dt=r.normal(b, L, D, dtype=io, scale=0.7, wide=wide),
             A=-(1.0 + torch.arange(N, device="cuda")) * torch.exp(r.normal(D, N, scale=0.1)),
             B=bc[..., :G * N].unflatten(-1, (G, N)), C=bc[..., G * N:].unflatten(-1, (G, N)),
             D=r.normal(D) if skip else None,
             z=r.normal(b, L, D, dtype=io, wide=wide) if z else None,
             dt_bias=r.normal(D, scale=0.5) - 4.0 if bias else None,
             h0=r.normal(b, D, N) if h0 else None)
    return s, r.normal(b, L, D, dtype=io, wide=wide), r.normal(b, D, N)


def norm_inputs(rows, D, dtype, seed=0, wide=0, bias=True, gate="input"):
    r, io = Draw(seed), DTYPES[dtype]
    shape = rows if isinstance(rows, tuple) else (rows,)
    return dict(x=r.normal(*shape, D, dtype=io, scale=1.5, wide=wide),
                weight=1.0 + r.normal(D, scale=0.3), bias=r.normal(D) if bias else None,
                z=None if gate == "none" else r.normal(*shape, D, dtype=io, wide=wide)), \
        r.normal(*shape, D, dtype=io, wide=wide)


def host(kw):
    return {k: (None if v is None else to64(v)) for k, v in kw.items()}
