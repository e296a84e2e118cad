"""The operators around the state space scan of a layer: the cases they are measured on,
and their plain forms.

Operators: the short causal convolution, the selective scan (a decay per channel and
state), the gated group norm, and the global gradient norm with clipping.  With `own`
false, run() computes a case from elementary torch operations in fp32; with `own` true it
makes the calls a user makes of the framework.  exact() restates each operator in float64.
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the convolution in front of a 2.7B-like Mamba-2 layer (80 heads of 64, one group
        # of 128 states: 5120 + 256 channels), reading its slice of the input projection
        dict(name="conv_prompt", op="conv", b=2, L=4096, D=5376, W=4, type="bf16",
             wide=5200, state=False, ragged=False),
        # the convolution's gradients in a 130M-like layer (24 heads of 64)
        dict(name="conv_train", op="conv_back", b=4, L=2048, D=1792, W=4, type="fp32",
             wide=1560, state=False, ragged=False),
        # one new token for each of 64 sequences
        dict(name="conv_token", op="conv_step", b=64, D=5376, W=4, type="bf16"),
        # prompts through a selective scan of 5120 channels, 16 states each
        dict(name="scan_prompt", op="scan", b=2, L=2048, D=5120, N=16, G=1, type="bf16",
             wide=5120, state=False, ragged=False),
        # one long document, few channels: the work is along the tokens
        dict(name="scan_long", op="scan", b=1, L=16384, D=1536, N=16, G=1, type="bf16",
             wide=1536, state=True, ragged=False),
        # padded prompts of different lengths (none and one token among them), odd sizes
        dict(name="scan_ragged", op="scan", b=4, L=509, D=771, N=13, G=3, type="fp32",
             wide=0, state=True, ragged=True),
        # the scan's gradients in training
        dict(name="scan_train", op="scan_back", b=4, L=1024, D=2048, N=16, G=1, type="bf16",
             wide=2048, state=False, ragged=False),
        # one new token for each of 64 sequences
        dict(name="scan_token", op="scan_step", b=64, D=5120, N=16, G=1, type="bf16"),
        # the norm in front of the output projection, gated by a slice of the projection
        dict(name="norm_prompt", op="norm", rows=8192, D=5120, G=1, type="bf16",
             gate="input", center=False, wide=5456),
        # its gradients, with eight groups
        dict(name="norm_train", op="norm_back", rows=8192, D=4096, G=8, type="bf16",
             gate="input", center=False, wide=0),
        # every gradient of a model of two 2.7B-like layers, kept in fp32
        dict(name="clip_model", op="clip", layers=2, width=2560, heads=80, type="fp32",
             max_norm=1.0),
        # two small layers with bf16 gradients that need no scaling
        dict(name="clip_small", op="clip", layers=2, width=160, heads=5, type="bf16",
             max_norm=1e6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_back", "conv_step", "scan", "scan", "scan_back",
                     "scan_step", "norm", "norm", "norm_back", "clip"])
    kind = rng.choice(["bf16", "fp32"])
    if op == "clip":
        heads = _log_int(rng, 1, 40)
        return dict(op=op, layers=_log_int(rng, 1, 6), width=32 * heads, heads=heads, type=kind,
                    max_norm=rng.choice([0.1, 1.0, 1e6]))
    if op in ("norm", "norm_back"):
        G = rng.choice([1, 1, 2, 3, 8])
        D = G * _log_int(rng, 8, 5120 // G)
        most = (20 << 20) if kind == "fp32" else (40 << 20)
        return dict(op=op, rows=_log_int(rng, 1, min(16384, most // D)), D=D, G=G, type=kind,
                    gate=rng.choice(["input", "output", "none"]),
                    center=rng.random() < 0.3, wide=rng.choice([0, 16, 37]))
    if op in ("conv_step", "scan_step"):
        case = dict(op=op, b=_log_int(rng, 1, 128), type=kind)
        if op == "conv_step":
            return dict(case, D=_log_int(rng, 16, 7168), W=rng.randint(2, 4))
        G = rng.choice([1, 1, 2, 3])
        return dict(case, D=G * _log_int(rng, 16, 5120 // G), N=rng.choice([16, 16, 8, 5, 32, 64]),
                    G=G)
    b = _log_int(rng, 1, 8)
    more = dict(type=kind, wide=rng.choice([0, 0, 24, 333]), state=rng.random() < 0.5,
                ragged=rng.random() < 0.4)
    if op in ("conv", "conv_back"):
        D = _log_int(rng, 16, 7168)
        most = (20 << 20) if op == "conv" and kind == "bf16" else (10 << 20)
        return dict(op=op, b=b, L=_log_int(rng, 1, max(1, min(16384, most // (b * D)))), D=D,
                    W=rng.randint(2, 4), **more)
    G = rng.choice([1, 1, 2, 3])
    D = G * _log_int(rng, 16, 4096 // G)
    N = rng.choice([16, 16, 16, 8, 5, 32, 64])
    most = ((128 << 20) if op == "scan_back" else (300 << 20)) // (b * D * N)
    return dict(op=op, b=b, L=_log_int(rng, 1, max(1, min(2048 if op == "scan_back" else 8192,
                                                          most))), D=D, N=N, G=G, **more)


def _lengths(case):
    """How many tokens of each padded sequence are real: all, none and one among them."""
    b, L = case["b"], case["L"]
    first = [L, 0, 1] if b > 2 else [max(1, L - L // 3), L]
    return [first[i] if i < len(first) else int(L * ((0.618 * i) % 1.0)) for i in range(b)]


def _shapes(case):
    """Parameter shapes of one model of gated state space layers."""
    dm, nh = case["width"], case["heads"]
    di, xbc = 64 * nh, 64 * nh + 256
    layer = [(di + xbc + nh, dm), (xbc, 4), (xbc,), (nh,), (nh,), (nh,), (di,), (dm, di), (dm,)]
    return layer * case["layers"] + [(dm,)]


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    io = _TYPES[case["type"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def rows(*shape):
        """[..., D] in the I/O type; with "wide", the last D columns of wider rows."""
        wide = case.get("wide", 0)
        return normal(*shape[:-1], wide + shape[-1], dtype=io)[..., wide:]

    op, s = case["op"], {"case": case}
    if op == "clip":
        s["grads"] = [normal(*n, scale=0.01, dtype=io) for n in _shapes(case)]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        return s
    D = case["D"]
    if op in ("norm", "norm_back"):
        s["x"] = normal(case["rows"], D, scale=2.0, dtype=io)
        s["weight"] = 1.0 + normal(D, scale=0.2)
        s["bias"] = normal(D, scale=0.2) if case["center"] else None
        s["z"] = None if case["gate"] == "none" else rows(case["rows"], D)
        s["gy"] = normal(case["rows"], D, dtype=io) if op == "norm_back" else None
        return s
    b, L = case["b"], case.get("L", 1)
    s["lengths"] = None
    if case.get("ragged"):
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if op.startswith("conv"):
        W = case["W"]
        s["weight"] = normal(D, W, scale=W ** -0.5)
        s["bias"] = normal(D, scale=0.2)
        if op == "conv_step":
            s["x"] = normal(b, D, dtype=io)
            s["state"] = normal(b, W - 1, D, dtype=io)
            return s
        s["x"] = rows(b, L, D)
        s["state"] = normal(b, W - 1, D, dtype=io) if case["state"] else None
        if op == "conv_back":
            s["gy"] = normal(b, L, D, dtype=io)
            s["gfinal"] = normal(b, W - 1, D, dtype=io) if case["state"] else None
        return s
    N, G = case["N"], case["G"]
    # step sizes of 1e-3 to 1e-1 before the token's own part, decays near -1 .. -N
    step = torch.exp(math.log(1e-3) + uniform(D) * math.log(100.0))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(torch.arange(N, device="cuda") + 1.0) * torch.exp(normal(D, N, scale=0.1))
    s["D"] = normal(D)
    seq = (b,) if op == "scan_step" else (b, L)
    s["u"] = normal(*seq, D, dtype=io)
    s["dt"] = normal(*seq, D, scale=0.5, dtype=io)
    s["z"] = rows(*seq, D)
    bc = normal(*seq, 2 * G * N + 8, dtype=io)  # one projection holds both, after 8 columns
    s["B"] = bc[..., 8:8 + G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., 8 + G * N:].unflatten(-1, (G, N))
    s["state"] = normal(b, D, N, scale=0.1) if case.get("state", True) else None
    if op == "scan_back":
        s["gy"] = normal(b, L, D, dtype=io)
        s["gfinal"] = normal(b, D, N, scale=0.1) if case["state"] else None
    return s


def work(case):
    op, size = case["op"], 2 if case["type"] == "bf16" else 4
    if op == "clip":
        n = sum(math.prod(shape) for shape in _shapes(case))
        return {"bytes": 2 * n * size, "flops": 3 * n}
    D = case["D"]
    if op in ("norm", "norm_back"):
        n, back = case["rows"] * D, op == "norm_back"
        gated = case["gate"] != "none"
        tensors = (3 + 2 * gated) if back else (2 + gated)
        return {"bytes": tensors * n * size + 4 * D * (1 + back),
                "flops": n * (20 if back else 10)}
    b = case["b"]
    tokens = sum(_lengths(case)) if case.get("ragged") else b * case.get("L", 1)
    out = b * case.get("L", 1)
    if op.startswith("conv"):
        W = case["W"]
        if op == "conv_step":
            return {"bytes": size * b * D * (2 + 2 * (W - 1)) + 4 * D * (W + 1),
                    "flops": b * D * (2 * W + 4)}
        states = size * b * D * (W - 1) * (1 + case["state"])
        if op == "conv":
            return {"bytes": size * D * (tokens + out) + states + 4 * D * (W + 1),
                    "flops": tokens * D * (2 * W + 4)}
        return {"bytes": size * D * (2 * tokens + out) + 2 * states + 8 * D * (W + 1),
                "flops": tokens * D * (6 * W + 12)}
    N, G = case["N"], case["G"]
    if op == "scan_step":
        return {"bytes": size * b * (4 * D + 2 * G * N) + 8 * b * D * N + 4 * D * (N + 2),
                "flops": b * D * (7 * N + 10)}
    states = 4 * b * D * N * (1 + case["state"])
    if op == "scan":
        return {"bytes": size * (tokens * (3 * D + 2 * G * N) + out * D) + states
                + 4 * D * (N + 2), "flops": tokens * D * (7 * N + 10)}
    return {"bytes": size * (tokens * (4 * D + 2 * G * N) + out * (3 * D + 2 * G * N))
            + 2 * states + 8 * D * (N + 2), "flops": tokens * D * (24 * N + 30)}


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import mamba_ssd_forward_gb300 as ssd
    case = s["case"]
    op = case["op"]
    if op == "clip":
        norm = ssd.clip_grad_norm(s["grads"], case["max_norm"], out=s["out"])
        return [norm] + s["out"]
    if op == "norm":
        return ssd.gated_norm_forward(s["x"], s["weight"], s["bias"], s["z"], groups=case["G"],
                                      gate=case["gate"], center=case["center"])
    if op == "norm_back":
        r = ssd.gated_norm_backward(s["x"], s["weight"], s["bias"], s["z"], s["gy"],
                                    groups=case["G"], gate=case["gate"], center=case["center"])
        return [r[k] for k in ("dx", "dz", "dweight", "dbias") if r[k] is not None]
    if op == "conv":
        return list(ssd.causal_conv_forward(s["x"], s["weight"], s["bias"], s["state"],
                                            lengths=s["lengths"]))
    if op == "conv_back":
        r = ssd.causal_conv_backward(s["x"], s["weight"], s["bias"], s["state"], s["gy"],
                                     s["gfinal"], lengths=s["lengths"])
        return [r[k] for k in ("dx", "dweight", "dbias", "dstate") if r[k] is not None]
    if op == "conv_step":
        return [ssd.causal_conv_step(s["x"], s["weight"], s["bias"], s["state"]), s["state"]]
    common = (s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["state"])
    if op == "scan_step":
        return [ssd.selective_scan_step(*common, dt_softplus=True), s["state"]]
    if op == "scan":
        return list(ssd.selective_scan_forward(*common, lengths=s["lengths"], dt_softplus=True))
    r = ssd.selective_scan_backward(*common, s["gy"], s["gfinal"], lengths=s["lengths"],
                                    dt_softplus=True)
    return [r[k] for k in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
            if r[k] is not None]


# --------------------------------------------------------- plain forms (fp32)

def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _dsilu(v):
    sig = 1.0 / (1.0 + torch.exp(-v))
    return sig * (1.0 + v * (1.0 - sig))


def _run_plain(s):
    op = s["case"]["op"]
    if op == "clip":
        return _plain_clip(s)
    if op in ("norm", "norm_back"):
        return _plain_norm(s)
    if op == "conv_step":
        return _plain_conv_step(s)
    if op.startswith("conv"):
        return _plain_conv(s)
    if op == "scan_step":
        return _plain_scan_step(s)
    return _plain_scan(s) if op == "scan" else _plain_scan_back(s)


def _plain_clip(s):
    total = torch.zeros((), device="cuda")
    for g in s["grads"]:
        f = g.float()
        total = total + (f * f).sum()
    norm = torch.sqrt(total)
    scale = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * scale)
    return [norm] + s["out"]


def _plain_norm(s, eps=1e-5):
    case, x, w = s["case"], s["x"].float(), s["weight"]
    io, gate, G = s["x"].dtype, case["gate"], case["G"]
    z = None if s["z"] is None else s["z"].float()
    rows, D = x.shape
    r = x * _silu(z) if gate == "input" else x
    rg = r.view(rows, G, D // G)
    if case["center"]:
        rg = rg - rg.mean(-1, keepdim=True)
    rstd = torch.rsqrt((rg * rg).mean(-1, keepdim=True) + eps)
    n = (rg * rstd).view(rows, D)
    v = n * w if s["bias"] is None else n * w + s["bias"]
    if s["gy"] is None:
        return (v * _silu(z) if gate == "output" else v).to(io)
    gy = s["gy"].float()
    gv = gy * _silu(z) if gate == "output" else gy
    dw, db = (gv * n).sum(0), gv.sum(0)
    gn = (gv * w).view(rows, G, D // G)
    ng = n.view(rows, G, D // G)
    gr = gn - ng * (gn * ng).mean(-1, keepdim=True)
    if case["center"]:
        gr = gr - gn.mean(-1, keepdim=True)
    gr = (gr * rstd).view(rows, D)
    dx = gr * _silu(z) if gate == "input" else gr
    outs = [dx.to(io)]
    if gate == "input":
        outs.append((gr * x * _dsilu(z)).to(io))
    elif gate == "output":
        outs.append((gy * v * _dsilu(z)).to(io))
    return outs + [dw] + ([] if s["bias"] is None else [db])


def _mask(s, L):
    """[b, L, 1] truth values: the real tokens (None = all)."""
    if s["lengths"] is None:
        return None
    return (torch.arange(L, device="cuda")[None, :] < s["lengths"][:, None])[..., None]


def _last_inputs(full, s, L, W):
    """The W - 1 inputs before each sequence's end, from [b, W - 1 + L, D]."""
    if s["lengths"] is None:
        return full[:, L:]
    at = s["lengths"].long()[:, None] + torch.arange(W - 1, device="cuda")
    return torch.gather(full, 1, at[..., None].expand(-1, -1, full.shape[2]))


def _plain_conv(s):
    case, io = s["case"], s["x"].dtype
    W, D, L, b = case["W"], case["D"], case["L"], case["b"]
    x, w, m = s["x"].float(), s["weight"], _mask(s, case["L"])
    if m is not None:
        x = torch.where(m, x, torch.zeros_like(x))
    first = torch.zeros(b, W - 1, D, device="cuda") if s["state"] is None else s["state"].float()
    full = torch.cat([first, x], 1)
    v = s["bias"] + sum(w[:, k] * full[:, k:k + L] for k in range(W))
    if case["op"] == "conv":
        y = _silu(v)
        if m is not None:
            y = torch.where(m, y, torch.zeros_like(y))
        return [y.to(io), _last_inputs(full, s, L, W).to(io)]
    g = s["gy"].float() * _dsilu(v)
    if m is not None:
        g = torch.where(m, g, torch.zeros_like(g))
    dfull = torch.zeros_like(full)
    dw = torch.empty_like(w)
    for k in range(W):
        dfull[:, k:k + L] += g * w[:, k]
        dw[:, k] = (g * full[:, k:k + L]).sum((0, 1))
    if s["gfinal"] is not None:
        if s["lengths"] is None:
            dfull[:, L:] += s["gfinal"].float()
        else:
            at = s["lengths"].long()[:, None] + torch.arange(W - 1, device="cuda")
            dfull.scatter_add_(1, at[..., None].expand(-1, -1, D), s["gfinal"].float())
    outs = [dfull[:, W - 1:].to(io), dw, g.sum((0, 1))]
    return outs if s["state"] is None else outs + [dfull[:, :W - 1].to(io)]


def _plain_conv_step(s):
    W = s["case"]["W"]
    full = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    v = s["bias"] + sum(s["weight"][:, k] * full[:, k] for k in range(W))
    s["state"].copy_(full[:, 1:])
    return [_silu(v).to(s["x"].dtype), s["state"]]


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_scan_step(s):
    G, N, io = s["case"]["G"], s["case"]["N"], s["u"].dtype
    b, D = s["u"].shape
    u = s["u"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    per = lambda t: t.float().repeat_interleave(D // G, dim=1)  # noqa: E731
    h = s["state"]
    h.copy_(torch.exp(delta[..., None] * s["A"]) * h + (delta * u)[..., None] * per(s["B"]))
    y = (h * per(s["C"])).sum(-1) + s["D"] * u
    return [(y * _silu(s["z"].float())).to(io), h]


def _scan_terms(s):
    """u, step sizes (zero past a sequence's end), A and B, C with the channels by group."""
    case = s["case"]
    b, L, D, N, G = (case[k] for k in ("b", "L", "D", "N", "G"))
    u = s["u"].float().view(b, L, G, D // G)
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    m = _mask(s, L)
    if m is not None:
        delta = torch.where(m, delta, torch.zeros_like(delta))
    h = (torch.zeros(b, D, N, device="cuda") if s["state"] is None else s["state"])
    return (u, delta.view(b, L, G, D // G), s["A"].view(G, D // G, N),
            s["B"].float()[:, :, :, None], s["C"].float()[:, :, :, None],
            h.view(b, G, D // G, N), m)


def _plain_scan(s):
    case, io = s["case"], s["u"].dtype
    b, L, D = case["b"], case["L"], case["D"]
    u, delta, A, B, C, h, m = _scan_terms(s)
    du = delta * u
    y = torch.empty_like(u)
    for t in range(L):
        h = torch.exp(delta[:, t, ..., None] * A) * h + du[:, t, ..., None] * B[:, t]
        y[:, t] = (h * C[:, t]).sum(-1)
    y = (y.view(b, L, D) + s["D"] * s["u"].float()) * _silu(s["z"].float())
    if m is not None:
        y = torch.where(m, y, torch.zeros_like(y))
    return [y.to(io), h.reshape(b, D, case["N"]).clone()]


def _plain_scan_back(s):
    case, io = s["case"], s["u"].dtype
    b, L, D, N, G = (case[k] for k in ("b", "L", "D", "N", "G"))
    u, delta, A, B, C, h, m = _scan_terms(s)
    du = delta * u
    hs = torch.empty(L + 1, *h.shape, device="cuda")
    hs[0] = h
    y = torch.empty_like(u)
    for t in range(L):
        h = torch.exp(delta[:, t, ..., None] * A) * h + du[:, t, ..., None] * B[:, t]
        hs[t + 1] = h
        y[:, t] = (h * C[:, t]).sum(-1)
    z, gy = s["z"].float(), s["gy"].float()
    if m is not None:
        gy = torch.where(m, gy, torch.zeros_like(gy))
    dz = gy * (y.view(b, L, D) + s["D"] * s["u"].float()) * _dsilu(z)
    go = gy * _silu(z)
    gt = go.view(b, L, G, D // G)
    g = (torch.zeros(b, D, N, device="cuda") if s["gfinal"] is None else s["gfinal"])
    g = g.view(b, G, D // G, N)
    gB_sum = torch.empty_like(u)  # sum over states of g B
    gah = torch.empty_like(u)     # sum over states of A g a h
    dB = torch.empty(b, L, G, N, device="cuda")
    dC = torch.empty(b, L, G, N, device="cuda")
    dA = torch.zeros_like(A)
    for t in reversed(range(L)):
        g = g + gt[:, t, ..., None] * C[:, t]
        dC[:, t] = (gt[:, t, ..., None] * hs[t + 1]).sum(2)
        dB[:, t] = (du[:, t, ..., None] * g).sum(2)
        gB_sum[:, t] = (g * B[:, t]).sum(-1)
        ga = g * torch.exp(delta[:, t, ..., None] * A)
        p = ga * hs[t]
        gah[:, t] = (p * A).sum(-1)
        dA = dA + (delta[:, t, ..., None] * p).sum(0)
        g = ga
    d_u = (delta * gB_sum).view(b, L, D) + go * s["D"]
    ddelta = (u * gB_sum + gah).view(b, L, D)
    d_raw = ddelta / (1.0 + torch.exp(-(s["dt"].float() + s["dt_bias"])))
    if m is not None:
        d_raw = torch.where(m, d_raw, torch.zeros_like(d_raw))
        d_u = torch.where(m, d_u, torch.zeros_like(d_u))
    outs = [d_u.to(io), d_raw.to(io), dA.reshape(D, N), dB.to(io), dC.to(io),
            (go * s["u"].float()).sum((0, 1)), dz.to(io), d_raw.sum((0, 1))]
    return outs if s["state"] is None else outs + [g.reshape(b, D, N).contiguous()]


# ------------------------------------------- the definitions again, in float64

def _f64(t):
    return None if t is None else t.detach().double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        return _exact_clip(s)
    if op.startswith("norm"):
        return _exact_norm(s)
    if op.startswith("conv"):
        return _exact_conv(s)
    return _exact_scan(s)


def _exact_clip(s):
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
    k = min(1.0, s["case"]["max_norm"] / (norm + 1e-6))
    return [torch.tensor(norm, dtype=torch.float64, device="cuda")] + \
        [g.double() * k for g in s["grads"]]


def _exact_norm(s, eps=1e-5):
    """The gradients are those of the definition by automatic differentiation."""
    case, back = s["case"], s["gy"] is not None
    leaf = {k: _f64(s[k]) for k in ("x", "z", "weight", "bias")}
    for t in leaf.values():
        if t is not None:
            t.requires_grad_(back)
    x, z, w, bias = (leaf[k] for k in ("x", "z", "weight", "bias"))
    a = x * z * torch.sigmoid(z) if case["gate"] == "input" else x
    a = a.unflatten(1, (case["G"], -1))
    mean = a.mean(2, keepdim=True) if case["center"] else 0.0
    var = ((a - mean) ** 2).mean(2, keepdim=True)
    v = ((a - mean) / torch.sqrt(var + eps)).flatten(1) * w
    if bias is not None:
        v = v + bias
    if case["gate"] == "output":
        v = v * z * torch.sigmoid(z)
    if not back:
        return v
    live = [t for t in (x, z, w, bias) if t is not None]
    return list(torch.autograd.grad(v, live, s["gy"].double()))


def _exact_conv(s):
    case, W, D, b = s["case"], s["case"]["W"], s["case"]["D"], s["case"]["b"]
    step = case["op"] == "conv_step"
    x = s["x"].double()[:, None] if step else s["x"].double()
    L = x.shape[1]
    n = [L] * b if s["lengths"] is None else s["lengths"].tolist()
    state = torch.zeros(b, W - 1, D, dtype=torch.float64, device="cuda") \
        if s["state"] is None else s["state"].double()
    w, bias = s["weight"].double(), s["bias"].double()
    back = case["op"] == "conv_back"
    leaf = [t.requires_grad_(back) for t in (x, w, bias, state)]
    ys, ends = [], []
    for i in range(b):  # one sequence at a time, its real tokens alone
        seq = torch.cat([state[i], x[i, :n[i]]])
        ends.append(seq[n[i]:])
        win = seq.unfold(0, W, 1) if n[i] else seq.new_zeros(0, D, W)
        v = (win * w).sum(-1) + bias
        ys.append(torch.cat([v * torch.sigmoid(v), v.new_zeros(L - n[i], D)]))
    y, end = torch.stack(ys), torch.stack(ends)
    if not back:
        return [y[:, 0] if step else y, end]
    gend = torch.zeros_like(end) if s["gfinal"] is None else s["gfinal"].double()
    grads = torch.autograd.grad([y, end], leaf, [s["gy"].double(), gend], allow_unused=True)
    grads = [torch.zeros_like(t) if g is None else g for g, t in zip(grads, leaf)]
    return grads[:3] if s["state"] is None else grads


def _prefix(a, v):
    """h_t = a_t h_{t-1} + v_t along axis 0 from zero, by doubling; overwrites both."""
    k = 1
    while k < a.shape[0]:
        v[k:] += a[k:] * v[:-k].clone()
        a[k:] *= a[:-k].clone()
        k *= 2
    return v


def _exact_scan(s):
    """One sequence and a slice of its channels at a time, by a scan over doubling spans."""
    case = s["case"]
    op, D, N, G, b = case["op"], case["D"], case["N"], case["G"], case["b"]
    step, back = op == "scan_step", op == "scan_back"
    seq = (lambda t: t.double()[:, None]) if step else (lambda t: t.double())
    u, raw, z = seq(s["u"]), seq(s["dt"]) + s["dt_bias"].double(), seq(s["z"])
    B, C = seq(s["B"]), seq(s["C"])
    L = u.shape[1]
    n = [L] * b if s["lengths"] is None else s["lengths"].tolist()
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    A, skip = s["A"].double(), s["D"].double()
    h0 = torch.zeros(b, D, N, dtype=torch.float64, device="cuda") \
        if s["state"] is None else s["state"].double()
    zero = torch.zeros_like
    y, end = zero(u), h0.clone()
    if back:
        gy = s["gy"].double()
        gend = zero(h0) if s["gfinal"] is None else s["gfinal"].double()
        sig = torch.sigmoid(z)
        go = gy * z * sig
        r = {k: zero(t) for k, t in (("du", u), ("ddt", u), ("dA", A), ("dB", B), ("dC", C),
                                     ("dD", skip), ("dz", u))}
        r["dh0"] = gend.clone()
    for i in range(b):
        T = n[i]
        if T == 0:
            continue
        per = D // G
        span = max(1, min(per, (96 << 20) // (T * N)))
        for grp in range(G):
            for lo in range(grp * per, (grp + 1) * per, span):
                c = slice(lo, min(lo + span, (grp + 1) * per))
                dl, uu = delta[i, :T, c], u[i, :T, c]
                a = torch.exp(dl[..., None] * A[c])
                v = (dl * uu)[..., None] * B[i, :T, grp, None, :]
                v[0] += a[0] * h0[i, c]
                h = _prefix(a.clone(), v)
                y[i, :T, c] = torch.einsum("tdn,tn->td", h, C[i, :T, grp])
                end[i, c] = h[-1]
                if not back:
                    continue
                # the adjoint runs the same recurrence backwards, its decay one token late
                q = go[i, :T, c][..., None] * C[i, :T, grp, None, :]
                q[-1] += gend[i, c]
                late = torch.cat([a[1:], zero(a[:1])])
                g = _prefix(late.flip(0), q.flip(0)).flip(0)
                before = torch.cat([h0[i, c][None], h[:-1]])
                p = g * a * before
                gB = torch.einsum("tdn,tn->td", g, B[i, :T, grp])
                r["du"][i, :T, c] = dl * gB + go[i, :T, c] * skip[c]
                r["ddt"][i, :T, c] = (uu * gB + (p * A[c]).sum(-1)) * torch.sigmoid(raw[i, :T, c])
                r["dA"][c] += torch.einsum("tdn,td->dn", p, dl)
                r["dB"][i, :T, grp] += torch.einsum("tdn,td->tn", g, dl * uu)
                r["dC"][i, :T, grp] += torch.einsum("tdn,td->tn", h, go[i, :T, c])
                r["dh0"][i, c] = a[0] * g[0]
        y[i, :T] += skip * u[i, :T]
        if back:
            r["dz"][i, :T] = gy[i, :T] * y[i, :T] * (sig * (1 + z * (1 - sig)))[i, :T]
            r["dD"] += (go[i, :T] * u[i, :T]).sum(0)
    if back:
        order = [r[k] for k in ("du", "ddt", "dA", "dB", "dC", "dD", "dz")]
        order.append(r["ddt"].sum((0, 1)))
        return order if s["state"] is None else order + [r["dh0"]]
    y = y * z * torch.sigmoid(z)
    return [y[:, 0] if step else y, end]
