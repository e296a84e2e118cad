"""Float64 references of the convolution and the selective scan in torch, all
sequences and channels at a time, for sizes at which the numpy oracle (one token
of one sequence after the other) takes too long.  Any device.  They are compared
with the oracle in test_layer_ref64_pins.py."""
import torch

F = torch.float64


def _f(t):
    return None if t is None else t.detach().to(F)


def _real(lengths, b, L, device):
    """[b, L, 1]: the tokens before each sequence's end."""
    n = torch.full((b,), L) if lengths is None else torch.tensor(lengths).clamp(0, L)
    n = n.to(device)
    return (torch.arange(L, device=device)[None] < n[:, None])[..., None], n


def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def _conv(x, weight, bias, state, lengths):
    """The masked inputs with the state in front, and the pre-activations."""
    x, w, bias, state = map(_f, (x, weight, bias, state))
    b, L, D = x.shape
    W = w.shape[1]
    real, n = _real(lengths, b, L, x.device)
    front = x.new_zeros(b, W - 1, D) if state is None else state
    full = torch.cat([front, torch.where(real, x, 0.0)], 1)
    v = sum(w[:, k] * full[:, k:k + L] for k in range(W))
    return full, v if bias is None else v + bias, w, real, n


def _last(n, W, D):
    """Indices into `full` of the inputs in front of each sequence's end."""
    return (n[:, None] + torch.arange(W - 1, device=n.device))[..., None].expand(-1, -1, D)


def causal_conv(x, weight, bias=None, state=None, lengths=None, act=True):
    full, v, w, real, n = _conv(x, weight, bias, state, lengths)
    y = torch.where(real, _silu(v) if act else v, 0.0)
    return y, torch.gather(full, 1, _last(n, w.shape[1], full.shape[2]))


def causal_conv_backward(x, weight, bias, state, gy, gfinal=None, lengths=None, act=True):
    full, v, w, real, n = _conv(x, weight, bias, state, lengths)
    W, L = w.shape[1], v.shape[1]
    g = torch.where(real, _f(gy) * _dsilu(v) if act else _f(gy), 0.0)
    dfull, dw = torch.zeros_like(full), torch.empty_like(w)
    for k in range(W):
        dfull[:, k:k + L] += w[:, k] * g
        dw[:, k] = (g * full[:, k:k + L]).sum((0, 1))
    if gfinal is not None:
        dfull.scatter_add_(1, _last(n, W, full.shape[2]), _f(gfinal))
    return {"dx": torch.where(real, dfull[:, W - 1:], 0.0), "dweight": dw,
            "dbias": g.sum((0, 1)), "dstate": dfull[:, :W - 1]}


def _scan(u, dt, A, B, C, D, z, dt_bias, h0, lengths, dt_softplus):
    u, dt, A, B, C, D, z, dt_bias, h0 = map(_f, (u, dt, A, B, C, D, z, dt_bias, h0))
    b, L, nd = u.shape
    real, _ = _real(lengths, b, L, u.device)
    raw = dt if dt_bias is None else dt + dt_bias
    s = torch.logaddexp(raw, torch.zeros_like(raw)) if dt_softplus else raw
    # a step of zero leaves the state alone
    s, u, z = (None if t is None else torch.where(real, t, 0.0) for t in (s, u, z))
    B, C = (torch.where(real[..., None], t, 0.0) for t in (B, C))
    h = u.new_zeros(b, nd, A.shape[1]) if h0 is None else h0
    return u, raw, s, A, B, C, u.new_zeros(nd) if D is None else D, z, h, real


def _of_channels(t, nd):
    """[b, G, N] for every channel of the groups: [b, D, N]."""
    return t.repeat_interleave(nd // t.shape[1], 1)


def _states(u, s, A, B, h):
    yield h
    for t in range(u.shape[1]):
        st = s[:, t, :, None]
        h = torch.exp(st * A) * h + st * u[:, t, :, None] * _of_channels(B[:, t], u.shape[2])
        yield h


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None,
                   dt_softplus=False):
    u, _, s, A, B, C, D, z, h, real = _scan(u, dt, A, B, C, D, z, dt_bias, h0, lengths,
                                            dt_softplus)
    y = torch.empty_like(u)
    for t, h in enumerate(_states(u, s, A, B, h), -1):
        if t >= 0:
            y[:, t] = (h * _of_channels(C[:, t], u.shape[2])).sum(2) + D * u[:, t]
    return torch.where(real, y if z is None else y * _silu(z), 0.0), h


def selective_scan_backward(u, dt, A, B, C, D, z, dt_bias, h0, gy, gfinal=None, lengths=None,
                            dt_softplus=False):
    u, raw, s, A, B, C, D, z, h, real = _scan(u, dt, A, B, C, D, z, dt_bias, h0, lengths,
                                              dt_softplus)
    b, L, nd = u.shape
    G, N = B.shape[2:]
    gy = torch.where(real, _f(gy), 0.0)
    hs = list(_states(u, s, A, B, h))
    o = gy if z is None else gy * _silu(z)
    r = {k: torch.zeros_like(t) for k, t in (("du", u), ("ddt", u), ("dz", u), ("dA", A),
                                             ("dB", B), ("dC", C))}
    g = torch.zeros_like(h) if gfinal is None else _f(gfinal)
    per = lambda t: t.view(b, G, nd // G, N).sum(2)  # noqa: E731
    for t in reversed(range(L)):
        Bt, Ct = (_of_channels(m[:, t], nd) for m in (B, C))
        st, ot = s[:, t, :, None], o[:, t, :, None]
        if z is not None:
            r["dz"][:, t] = gy[:, t] * ((hs[t + 1] * Ct).sum(2) + D * u[:, t]) * _dsilu(z[:, t])
        g = g + ot * Ct
        q = g * torch.exp(st * A)
        p = q * hs[t]
        gB = (g * Bt).sum(2)
        r["du"][:, t] = s[:, t] * gB + D * o[:, t]
        r["ddt"][:, t] = u[:, t] * gB + (A * p).sum(2)
        r["dA"] += (st * p).sum(0)
        r["dB"][:, t] = per(g * st * u[:, t, :, None])
        r["dC"][:, t] = per(hs[t + 1] * ot)
        g = q
    if dt_softplus:
        r["ddt"] = r["ddt"] * torch.sigmoid(raw)
    r["ddt"] = torch.where(real, r["ddt"], 0.0)
    r["du"] = torch.where(real, r["du"], 0.0)
    for k in ("dB", "dC"):
        r[k] = torch.where(real[..., None], r[k], 0.0)
    return {**r, "dD": (o * u).sum((0, 1)), "ddt_bias": r["ddt"].sum((0, 1)), "dh0": g}
