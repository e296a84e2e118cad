"""float64 definitions of the operators around a language model's blocks, in torch on
any device, and how far a kernel's result may be off: bounds from the roundings it
makes, written down before it first ran.

A rounding to nearest is off by at most half a step, eps / 2 of the value.  The tensor
cores cut a sum at 24 bits when they add to it, up to 2^-23 of it each time."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


# ------------------------------------------------------ residual and norm

def add_norm(x, residual, weight, eps=1e-5):
    t = x.double() + (0.0 if residual is None else residual.double())
    rstd = 1.0 / torch.sqrt((t ** 2).mean(-1, keepdim=True) + eps)
    return t * rstd * weight.double(), t


def add_norm_backward(total, weight, gy, gtotal, eps=1e-5):
    """By the quotient rule, a channel at a time in the formula's own terms:
    dy_i/dt_j = w_i (delta_ij r - t_i t_j r^3 / D), r = 1 / sqrt(mean t^2 + eps)."""
    t, g = total.double(), gy.double()
    D = t.shape[-1]
    r = ((t ** 2).mean(-1, keepdim=True) + eps) ** -0.5
    gw = g * weight.double()
    dt = gw * r - t * (gw * t).sum(-1, keepdim=True) * r ** 3 / D
    if gtotal is not None:
        dt = dt + gtotal.double()
    dw = (g * t * r).reshape(-1, D).sum(0)
    return dt, dw


def norm_bound(D, dtype):
    """Relative: the output's rounding, and that of the sum of D squares (half of it, for
    the root), the root and three products."""
    return HALF[dtype] + (D / 2 + 8) * 2.0 ** -24


# ---------------------------------------------------------- cross entropy

def cross_entropy(x, weight, targets, ignore=-100):
    """loss, lse, both zero for tokens without a target, and which have one."""
    d, V = x.shape[-1], weight.shape[0]
    xs, t = x.reshape(-1, d).double(), targets.reshape(-1)
    live = t != ignore
    z = torch.where(live[:, None], xs, 0.0) @ weight.double().t()
    lse = torch.logsumexp(z, 1)
    bad = live & ((t < 0) | (t >= V))
    zt = z.gather(1, torch.where(live & ~bad, t, 0)[:, None])[:, 0]
    loss = torch.where(bad, math.nan, lse - zt)
    zero = torch.zeros_like(lse)
    return torch.where(live, loss, zero), torch.where(live, lse, zero), live


def cross_entropy_backward(x, weight, targets, g, ignore=-100):
    """dx, dweight, and the sums of the absolute values of their terms; g: a factor for
    each token."""
    d = x.shape[-1]
    xs, t, w = x.reshape(-1, d).double(), targets.reshape(-1), weight.double()
    live = t != ignore
    xs = torch.where(live[:, None], xs, 0.0)
    z = xs @ w.t()
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    p[torch.arange(len(t), device=t.device), torch.where(live, t, 0)] -= 1.0
    p *= torch.where(live, g.reshape(-1).double(), 0.0)[:, None]
    return (p @ w).reshape(x.shape), p.t() @ xs, (p.abs() @ w.abs()).reshape(x.shape), \
        p.abs().t() @ xs.abs()


def logit_bound(x, weight, dtype, live):
    """Of a logit, absolute: bf16 products are exact and d / 16 cut sums follow; fp32
    operands have 22 bits (2^-23 each, 2^-22 what is dropped), segments of 16 cut sums,
    and 3 d / 256 segments."""
    d = x.shape[-1]
    xs = x.reshape(-1, d).double()[live.reshape(-1)]
    if not len(xs):
        return 0.0
    top = float((xs.abs() @ weight.double().abs().t()).max())
    if dtype == torch.bfloat16:
        return top * (d / 16 + 4) * 2.0 ** -23
    return top * (2.0 ** -21 + (16 + 3 * d / 256 + 4) * 2.0 ** -23)


def loss_bound(z_off, V, loss):
    """Twice a logit's (lse and the target's), exponentials off by 2^-21 of each, sums
    of V / 128 runs of 128, and the result's own roundings."""
    return 2 * z_off + 2.0 ** -20 + (V / 128 + 128) * 2.0 ** -24 + loss.abs() * 2.0 ** -22


def grad_bound(z_off, lse_top, terms, count, value, dtype):
    """Each term is off by its operand's rounding (bf16: 2^-8 of dz; fp32 planes: 2^-21
    of the product), by exp of the logit's and lse's errors, and lse's own rounding;
    `count` terms are summed."""
    each = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20
    each += 2 * z_off + 2.0 ** -19 + lse_top * 2.0 ** -22
    cut = (count / 16 + 8) if dtype == torch.bfloat16 else (24 + 3 * count / 256)
    return terms * (each + cut * 2.0 ** -23) + value.abs() * HALF[dtype] * 2 + 1e-30


# ---------------------------------------------------------- orthogonalisation

def orthogonalize(update, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """Through the singular values: a step maps each by a s + b s^3 + c s^5."""
    a, b, c = coefficients
    u, s, vh = torch.linalg.svd(update.double(), full_matrices=False)
    s = s / ((s ** 2).sum(-1, keepdim=True).sqrt() + eps)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return u * s[..., None, :] @ vh


def orth_bound(dtype, update, steps=5, coefficients=(3.4445, -4.7750, 2.0315)):
    """Relative in the 2-norm, for operands of 11 bits (22 for an fp32 result):

    the result's rounding; X itself, of 22 bits, rounded before each step and after
    the last, small values enlarged a = 3.4445 times by each step that follows (a sum over
    the steps); and the roundings of A, B and X as operands of B X, of size |b| + 2 |c|
    (A's) + 2 (|b| - |c|) (B's and X's) = 14.3 at singular values of 1.  Of 16 x 16 values
    and more these are taken as independent (a root of squares over the entries and the
    steps); of fewer they may all point one way, and then grow with the slope of the
    steps that follow, at the update's own singular values."""
    a, b, c = coefficients
    unit = 2.0 ** (-12 if dtype == torch.bfloat16 else -23)
    size = abs(b) + 2 * abs(c) + 2 * abs(abs(b) - abs(c))
    carried = 2.0 ** -23 * sum(max(a, 1.0) ** k for k in range(steps + 1))
    if min(update.shape[-2:]) >= 16:
        return HALF[dtype] + carried + math.sqrt(steps) * size * unit / math.sqrt(3)
    s = torch.linalg.svdvals(update.double())
    s = s / ((s ** 2).sum(-1, keepdim=True).sqrt() + 1e-7)
    off = torch.zeros_like(s)
    for _ in range(steps):
        off = off * (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs() + size * unit
        s = a * s + b * s ** 3 + c * s ** 5
    worst = (off ** 2).sum(-1).sqrt() / (s ** 2).sum(-1).sqrt()
    return HALF[dtype] + carried + float(worst.max())
