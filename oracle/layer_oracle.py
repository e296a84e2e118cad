"""Float64 restatements of the operators around the scan: the short causal
convolution, the selective scan, the gated group norm and gradient clipping.

TEST INFRASTRUCTURE ONLY (see the package docstring).  numpy, one token after
the other where the operator is a recurrence; the gradients are the formulas
written out, pinned by central differences of the forwards.

`lengths` (a list, or None) gives each sequence's real tokens; what the inputs
hold past them is never read.
"""
from __future__ import annotations

import numpy as np

F = np.float64


def _f(t):
    return None if t is None else np.asarray(t, F)


def _sigmoid(v):
    v = np.clip(v, -700.0, 700.0)
    return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * _sigmoid(v)


def dsilu(v):
    s = _sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def _lens(lengths, b, L):
    return [L] * b if lengths is None else [int(min(max(n, 0), L)) for n in lengths]


# ------------------------------------------------------ causal convolution

def causal_conv(x, weight, bias=None, state=None, lengths=None, act=True):
    """y, final_state; x [b, L, D], weight [D, W], state [b, W - 1, D]."""
    x, w, bias, state = _f(x), _f(weight), _f(bias), _f(state)
    b, L, D = x.shape
    W = w.shape[1]
    y, final = np.zeros((b, L, D)), np.zeros((b, W - 1, D))
    for i, n in enumerate(_lens(lengths, b, L)):
        rows = list(np.zeros((W - 1, D)) if state is None else state[i]) + list(x[i, :n])
        for t in range(n):
            v = sum(w[:, k] * rows[t + k] for k in range(W))
            v = v if bias is None else v + bias
            y[i, t] = silu(v) if act else v
        final[i] = np.array(rows[n:n + W - 1])
    return y, final


def causal_conv_backward(x, weight, bias, state, gy, gfinal=None, lengths=None, act=True):
    x, w, bias, state, gy, gfinal = map(_f, (x, weight, bias, state, gy, gfinal))
    b, L, D = x.shape
    W = w.shape[1]
    dx, dw, db = np.zeros((b, L, D)), np.zeros((D, W)), np.zeros(D)
    dstate = np.zeros((b, W - 1, D))
    for i, n in enumerate(_lens(lengths, b, L)):
        rows = list(np.zeros((W - 1, D)) if state is None else state[i]) + list(x[i, :n])
        drows = np.zeros((W - 1 + n, D))
        for t in range(n):
            v = sum(w[:, k] * rows[t + k] for k in range(W))
            v = v if bias is None else v + bias
            g = gy[i, t] * dsilu(v) if act else gy[i, t]
            db += g
            for k in range(W):
                dw[:, k] += g * rows[t + k]
                drows[t + k] += g * w[:, k]
        if gfinal is not None:
            drows[n:] += gfinal[i]
        dstate[i], dx[i, :n] = drows[:W - 1], drows[W - 1:]
    return {"dx": dx, "dweight": dw, "dbias": db, "dstate": dstate}


# ----------------------------------------------------------- selective scan

def _scan_setup(u, dt, A, B, C, D, z, dt_bias, h0, dt_softplus):
    u, dt, A, B, C, D, z, dt_bias, h0 = map(_f, (u, dt, A, B, C, D, z, dt_bias, h0))
    b, L, nd = u.shape
    per = nd // B.shape[2]
    raw = dt if dt_bias is None else dt + dt_bias
    s = np.logaddexp(raw, 0.0) if dt_softplus else raw
    D = np.zeros(nd) if D is None else D
    h0 = np.zeros((b, nd, A.shape[1])) if h0 is None else h0
    return u, raw, s, A, np.repeat(B, per, 2), np.repeat(C, per, 2), D, z, h0, per


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None,
                   dt_softplus=False):
    """y [b, L, D], final_state [b, D, N], by the recurrence."""
    u, _, s, A, B, C, D, z, h0, _ = _scan_setup(u, dt, A, B, C, D, z, dt_bias, h0, dt_softplus)
    y, final = np.zeros(u.shape), h0.copy()
    for i, n in enumerate(_lens(lengths, *u.shape[:2])):
        h = h0[i].copy()
        for t in range(n):
            h = np.exp(s[i, t][:, None] * A) * h + (s[i, t] * u[i, t])[:, None] * B[i, t]
            y[i, t] = (h * C[i, t]).sum(1) + D * u[i, t]
            if z is not None:
                y[i, t] *= silu(z[i, t])
        final[i] = h
    return y, final


def selective_scan_backward(u, dt, A, B, C, D, z, dt_bias, h0, gy, gfinal=None, lengths=None,
                            dt_softplus=False):
    has_z, gy, gfinal = z is not None, _f(gy), _f(gfinal)
    G = np.asarray(B).shape[2]
    u, raw, s, A, B, C, D, z, h0, per = _scan_setup(u, dt, A, B, C, D, z, dt_bias, h0,
                                                    dt_softplus)
    b, L, nd = u.shape
    N = A.shape[1]
    r = {k: np.zeros((b, L, nd)) for k in ("du", "ddt", "dz")}
    r.update(dA=np.zeros((nd, N)), dB=np.zeros((b, L, G, N)), dC=np.zeros((b, L, G, N)),
             dD=np.zeros(nd), dh0=np.zeros((b, nd, N)))
    for i, n in enumerate(_lens(lengths, b, L)):
        hs = [h0[i]]
        for t in range(n):
            hs.append(np.exp(s[i, t][:, None] * A) * hs[-1]
                      + (s[i, t] * u[i, t])[:, None] * B[i, t])
        g = np.zeros((nd, N)) if gfinal is None else gfinal[i].copy()
        for t in reversed(range(n)):
            o = gy[i, t]
            if has_z:
                yv = (hs[t + 1] * C[i, t]).sum(1) + D * u[i, t]
                r["dz"][i, t] = o * yv * dsilu(z[i, t])
                o = o * silu(z[i, t])
            e = np.exp(s[i, t][:, None] * A)
            g = g + o[:, None] * C[i, t]
            p = g * e * hs[t]
            gB = (g * B[i, t]).sum(1)
            r["du"][i, t] = s[i, t] * gB + D * o
            ds = u[i, t] * gB + (A * p).sum(1)
            r["ddt"][i, t] = ds * _sigmoid(raw[i, t]) if dt_softplus else ds
            r["dA"] += s[i, t][:, None] * p
            r["dB"][i, t] = (g * (s[i, t] * u[i, t])[:, None]).reshape(G, per, N).sum(1)
            r["dC"][i, t] = (hs[t + 1] * o[:, None]).reshape(G, per, N).sum(1)
            r["dD"] += o * u[i, t]
            g = g * e
        r["dh0"][i] = g
    r["ddt_bias"] = r["ddt"].sum((0, 1))
    return r


# -------------------------------------------------------- gated group norm

def _normed(x, z, groups, eps, gate, center):
    rows, D = x.shape
    r = (x * silu(z) if gate == "input" else x).reshape(rows, groups, D // groups)
    if center:
        r = r - r.mean(2, keepdims=True)
    rstd = 1.0 / np.sqrt((r * r).mean(2, keepdims=True) + eps)
    return r * rstd, rstd


def gated_norm(x, weight, bias=None, z=None, groups=1, eps=1e-5, gate="input", center=False):
    """y [rows, D]."""
    x, w, bias, z = map(_f, (x, weight, bias, z))
    n, _ = _normed(x, z, groups, eps, gate, center)
    v = n.reshape(x.shape) * w + (0.0 if bias is None else bias)
    return v * silu(z) if gate == "output" else v


def gated_norm_backward(x, weight, bias, z, gy, groups=1, eps=1e-5, gate="input", center=False):
    x, w, bias, z, gy = map(_f, (x, weight, bias, z, gy))
    n, rstd = _normed(x, z, groups, eps, gate, center)
    flat = n.reshape(x.shape)
    gv = gy * silu(z) if gate == "output" else gy
    q = (gv * w).reshape(n.shape)
    gr = q - n * (q * n).mean(2, keepdims=True)
    if center:
        gr = gr - q.mean(2, keepdims=True)
    gr = (gr * rstd).reshape(x.shape)
    out = {"dweight": (gv * flat).sum(0), "dbias": gv.sum(0), "dx": gr, "dz": None}
    if gate == "input":
        out["dx"], out["dz"] = gr * silu(z), gr * x * dsilu(z)
    elif gate == "output":
        out["dz"] = gy * (flat * w + (0.0 if bias is None else bias)) * dsilu(z)
    return out


# -------------------------------------------- gradient norm and clipping

def clip_grad_norm(grads, max_norm, eps=1e-6):
    """norm, scaled tensors."""
    grads = [_f(g) for g in grads]
    norm = np.sqrt(sum((g * g).sum() for g in grads))
    return norm, [g * min(1.0, max_norm / (norm + eps)) for g in grads]
