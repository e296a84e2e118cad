"""The operators around the blocks of a language model: the cases they are measured on, and
their plain forms.

Operators: the residual's addition with the norm in front of a block (its gradients, and its
output in 8 bits with scales), the cross entropy over a large vocabulary from the last hidden
states without keeping the logits (with its gradients), and the orthogonalisation of an update
by Newton-Schulz products.  With `own` false, run() computes a case from elementary torch
operations in fp32; with `own` true it makes the calls a user makes of the framework.  exact()
restates each operator in float64.
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
_E4M3 = torch.float8_e4m3fn
_TOP = 448.0  # the largest e4m3 value
_STEPS, _COEFFS, _TINY = 5, (3.4445, -4.7750, 2.0315), 1e-7


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the norm in front of a 2.7B-like block over two prompts, the residual stream in fp32
        dict(name="norm_prompt", op="norm", rows=8192, D=2560, type="bf16", stream="fp32"),
        # its gradients in training, the residual stream in the activations' type
        dict(name="norm_train", op="norm_back", rows=8192, D=2560, type="bf16", stream="bf16"),
        # prompts whose projection runs in 8 bits: a scale for each 128 channels of a token
        dict(name="norm8_prompt", op="norm8", rows=16384, D=5120, block=128, type="bf16",
             stream="bf16"),
        # one new token for each of 64 sequences, a scale for each token
        dict(name="norm8_token", op="norm8", rows=64, D=2560, block=0, type="bf16",
             stream="fp32"),
        # a training step's loss and gradients: 8192 tokens, a 2.7B-like model's width
        dict(name="loss_train", op="loss_back", rows=8192, D=2560, V=50280, type="bf16",
             ignored=0.0, spread=1.0),
        # scoring 2048 tokens with a 130M-like model
        dict(name="loss_score", op="loss", rows=2048, D=768, V=50280, type="bf16", ignored=0.0,
             spread=3.0),
        # fp32 training of a small model of odd sizes, a third of the tokens without a target
        dict(name="loss_odd", op="loss_back", rows=1021, D=771, V=32003, type="fp32",
             ignored=0.33, spread=2.0),
        # the loss of the last token of each of 5 sequences
        dict(name="loss_token", op="loss", rows=5, D=2560, V=50280, type="bf16", ignored=0.0,
             spread=1.0),
        # the update of a 2.7B-like block's input projection
        dict(name="orth_projection", op="orth", k=1, m=10576, n=2560, type="bf16", to="bf16"),
        # those of the output projections of a 130M-like model's 24 blocks, together
        dict(name="orth_blocks", op="orth", k=24, m=768, n=1536, type="bf16", to="bf16"),
        # an update of odd sizes, kept in fp32
        dict(name="orth_odd", op="orth", k=1, m=509, n=771, type="fp32", to="fp32"),
        # the input projection of a small block: the products are tiny, latency counts
        dict(name="orth_small", op="orth", k=1, m=644, n=128, type="fp32", to="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "norm8", "loss", "loss_back", "orth", "orth"])
    kind = rng.choice(["bf16", "fp32"])
    if op == "orth":
        k = rng.choice([1, 1, 2, 6])
        m, n = _log_int(rng, 16, 5120), _log_int(rng, 16, 5120)
        while k * m * n * min(m, n) > 10576 * 2560 * 2560:
            m, n = (m + 1) // 2, (n + 1) // 2
        return dict(op=op, k=k, m=m, n=n, type=kind, to=rng.choice(["bf16", "fp32"]))
    if op in ("loss", "loss_back"):
        rows, D, V = _log_int(rng, 1, 8192), _log_int(rng, 64, 2560), _log_int(rng, 257, 65536)
        if rng.random() < 0.5:
            D, V = -(-D // 8) * 8, -(-V // 8) * 8
        return dict(op=op, rows=rows, D=D, V=V, type=kind,
                    ignored=rng.choice([0.0, 0.0, 0.33, 0.8]), spread=rng.choice([1.0, 3.0, 8.0]))
    D = _log_int(rng, 16, 5120)
    case = dict(op=op, rows=_log_int(rng, 1, min(16384, (80 << 20) // D)), D=D, type=kind,
                stream="fp32" if kind == "fp32" else rng.choice(["bf16", "fp32"]))
    if op == "norm8":
        case["block"] = rng.choice([0, 32, 64, 128])
    return case


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, io = case["op"], _TYPES[case["type"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if op == "orth":
        # a few strong directions and a floor of noise, as gradients of projections have
        k, m, n = case["k"], case["m"], case["n"]
        r = max(1, min(m, n) // 8)
        falloff = torch.exp(-3.0 * torch.arange(r, device="cuda") / r)
        s["update"] = (1e-3 * ((normal(k, m, r) * falloff) @ normal(k, r, n) / math.sqrt(r)
                               + 0.05 * normal(k, m, n))).to(io)
        return s
    rows, D = case["rows"], case["D"]
    if op in ("loss", "loss_back"):
        V = case["V"]
        s["x"] = normal(rows, D, dtype=io)
        s["weight"] = normal(V, D, scale=case["spread"] / math.sqrt(D), dtype=io)
        t = torch.randint(0, V, (rows,), generator=g, device="cuda")
        u = torch.rand(rows, generator=g, device="cuda")
        s["targets"] = torch.where(u < case["ignored"], -100, t)
        return s
    stream = _TYPES[case["stream"]]
    s["weight"] = 1.0 + normal(D, scale=0.2)
    if op == "norm_back":
        s["total"] = normal(rows, D, scale=2.0, dtype=stream)
        s["gy"] = normal(rows, D, dtype=io)
        s["gtotal"] = normal(rows, D, dtype=stream)
        return s
    s["x"] = normal(rows, D, dtype=io)
    s["residual"] = normal(rows, D, scale=2.0, dtype=stream)
    return s


def work(case):
    op, size = case["op"], 2 if case["type"] == "bf16" else 4
    if op == "orth":
        m, n = sorted((case["m"], case["n"]))
        per = m * m * n + m * m * m + 2 * m * m * n  # two symmetric products and a full one
        return {"bytes": case["k"] * m * n * (size + (2 if case["to"] == "bf16" else 4)),
                "flops": case["k"] * _STEPS * per}
    rows, D = case["rows"], case["D"]
    if op in ("loss", "loss_back"):
        V, live = case["V"], rows * (1.0 - case["ignored"])
        inputs = size * (live * D + V * D) + 8 * rows
        if op == "loss":
            return {"bytes": inputs + 4 * rows, "flops": 2 * live * V * D}
        # forward; then the logits again and two products
        return {"bytes": 2 * inputs + size * (rows * D + V * D), "flops": 8 * live * V * D}
    wide = 2 if case["stream"] == "bf16" else 4
    if op == "norm_back":
        apart = size if case["stream"] != case["type"] else 0  # dx apart from the residual's
        return {"bytes": rows * D * (size + 3 * wide + apart) + 8 * D, "flops": 12 * rows * D}
    out = size if op == "norm" else 1 + 4 / (case["block"] or D)
    return {"bytes": rows * D * (size + 2 * wide + out) + 4 * D, "flops": 6 * rows * D}


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import mamba_ssd_forward_gb300 as ssd
    case = s["case"]
    op = case["op"]
    if op == "orth":
        return ssd.orthogonalize(s["update"], dtype=_TYPES[case["to"]])
    if op == "loss":
        return list(ssd.linear_cross_entropy_forward(s["x"], s["weight"], s["targets"]))
    if op == "loss_back":
        loss, lse = ssd.linear_cross_entropy_forward(s["x"], s["weight"], s["targets"],
                                                     reduction="mean")
        r = ssd.linear_cross_entropy_backward(s["x"], s["weight"], s["targets"], lse,
                                              reduction="mean")
        return [loss, r["dx"], r["dweight"]]
    if op == "norm":
        return list(ssd.add_norm_forward(s["x"], s["residual"], s["weight"]))
    if op == "norm8":
        return list(ssd.add_norm_quantized(s["x"], s["residual"], s["weight"],
                                           block=case["block"]))
    r = ssd.add_norm_backward(s["total"], s["weight"], s["gy"], s["gtotal"])
    return [r["dx"], r["dresidual"], r["dweight"]]


# --------------------------------------------------------- plain forms (fp32)

def _run_plain(s):
    op = s["case"]["op"]
    if op == "orth":
        return _plain_orth(s)
    if op in ("loss", "loss_back"):
        return _plain_loss(s)
    return _plain_norm_back(s) if op == "norm_back" else _plain_norm(s)


def _plain_norm(s, eps=1e-5):
    case, x = s["case"], s["x"]
    t = x.float() + s["residual"].float()
    y = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + eps) * s["weight"]
    total = t.to(s["residual"].dtype)
    if case["op"] == "norm":
        return [y.to(x.dtype), total]
    rows, D = x.shape
    c = case["block"] or D
    parts = -(-D // c)
    padded = torch.zeros(rows, parts * c, device="cuda")
    padded[:, :D] = y
    padded = padded.view(rows, parts, c)
    top = padded.abs().amax(-1)
    factor = torch.where(top > 0, _TOP / top, torch.zeros_like(top))
    q = (padded * factor[..., None]).view(rows, parts * c)[:, :D]
    return [q.to(_E4M3), top / _TOP, total]


def _plain_norm_back(s, eps=1e-5):
    t, gy, w = s["total"].float(), s["gy"].float(), s["weight"]
    rstd = torch.rsqrt((t * t).mean(-1, keepdim=True) + eps)
    n = t * rstd
    g = gy * w
    dt = rstd * (g - n * (g * n).mean(-1, keepdim=True)) + s["gtotal"].float()
    return [dt.to(s["gy"].dtype), dt.to(s["total"].dtype), (gy * n).sum(0)]


def _plain_loss(s):
    case, io = s["case"], s["x"].dtype
    x, w, targets = s["x"].float(), s["weight"].float(), s["targets"]
    live = targets >= 0
    at = torch.where(live, targets, 0)[:, None]
    z = x @ w.t()
    top = z.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(-1, keepdim=True))
    loss = torch.where(live, (lse - z.gather(1, at))[:, 0], 0.0)
    if case["op"] == "loss":
        return [loss, torch.where(live, lse[:, 0], 0.0)]
    share = 1.0 / torch.clamp(live.sum(), min=1).float()
    dz = torch.exp(z - lse)
    dz.scatter_add_(1, at, torch.full_like(lse, -1.0))
    dz *= live[:, None] * share
    return [loss.sum() * share, (dz @ w).to(io), (dz.t() @ x).to(io)]


def _plain_orth(s):
    case, x = s["case"], s["update"].float()
    a, b, c = _COEFFS
    tall = case["m"] > case["n"]
    x = x.transpose(1, 2) if tall else x
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + _TINY)
    for _ in range(_STEPS):
        sq = x @ x.transpose(1, 2)
        x = a * x + (b * sq + c * (sq @ sq)) @ x
    return (x.transpose(1, 2) if tall else x).to(_TYPES[case["to"]]).contiguous()


# ------------------------------------------- the definitions again, in float64

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "orth":
        return _exact_orth(s)
    if op in ("loss", "loss_back"):
        return _exact_loss(s)
    return _exact_norm(s)


def _exact_norm(s, eps=1e-5):
    """The gradients by automatic differentiation; values in 8 bits before their rounding."""
    case, w = s["case"], s["weight"].double()
    back = case["op"] == "norm_back"
    total = s["total"].double() if back else s["x"].double() + s["residual"].double()
    leaf = [total.requires_grad_(back), w.requires_grad_(back)]
    y = total / torch.sqrt(total.pow(2).mean(1, keepdim=True) + eps) * w
    if back:
        dt, dw = torch.autograd.grad([y, total], leaf, [s["gy"].double(), s["gtotal"].double()])
        return [dt, dt, dw]
    if case["op"] == "norm":
        return [y, total]
    block = case["block"] or case["D"]
    scaled, scales = [], []
    for part in y.split(block, dim=1):
        scale = part.abs().max(dim=1, keepdim=True).values / _TOP
        scales.append(scale)
        scaled.append(part / torch.where(scale == 0, 1.0, scale))
    return [torch.cat(scaled, 1), torch.cat(scales, 1), total]


def _exact_loss(s):
    """The gradients by the definition's derivative, a few thousand words at a time."""
    case = s["case"]
    keep = torch.nonzero(s["targets"] >= 0).flatten()
    x, w, t = s["x"][keep].double(), s["weight"].double(), s["targets"][keep]
    n, step = keep.numel(), 8192
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
    for lo in range(0, case["V"], step):
        lse = torch.logaddexp(lse, torch.logsumexp(x @ w[lo:lo + step].t(), 1))
    loss = lse - (x * w[t]).sum(1)
    if case["op"] == "loss":
        out = torch.zeros(2, case["rows"], dtype=torch.float64, device="cuda")
        out[0, keep], out[1, keep] = loss, lse
        return [out[0], out[1]]
    dw, dx = torch.zeros_like(w), torch.zeros_like(x)
    for lo in range(0, case["V"], step):
        part = w[lo:lo + step]
        p = torch.exp(x @ part.t() - lse[:, None])
        dx += p @ part
        dw[lo:lo + step] = p.t() @ x
    dx -= w[t]
    dw.index_add_(0, t, x, alpha=-1.0)
    whole = torch.zeros(case["rows"], case["D"], dtype=torch.float64, device="cuda")
    whole[keep] = dx
    share = 1.0 / max(1, n)
    return [loss.sum() * share, whole * share, dw * share]


def _exact_orth(s):
    """By the singular values' polynomial: each step maps them and keeps the vectors.  Written
    as products of the Gram matrix, whose powers commute, so no decomposition is needed."""
    a, b, c = _COEFFS
    out = []
    for g in s["update"].double().unbind(0):
        x = g / (torch.linalg.matrix_norm(g) + _TINY)
        for _ in range(_STEPS):
            if x.shape[0] <= x.shape[1]:
                gram = x @ x.mT
                gx = gram @ x
                x = a * x + b * gx + c * (gram @ gx)
            else:
                gram = x.mT @ x
                xg = x @ gram
                x = a * x + b * xg + c * (xg @ gram)
        out.append(x)
    return torch.stack(out)
