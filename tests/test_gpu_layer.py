"""GPU parity of the operators around the scan against their float64 oracle:
the causal convolution, the selective scan, the gated norm and gradient
clipping; forward, backward and single token, at the sizes, strides, lengths
and values where they can go wrong.  Tolerances: layer_cases.py."""
import numpy as np
import pytest
import torch

from layer_cases import (DTYPES, Draw, close, conv_inputs, host, lengths_of, norm_inputs,
                         scan_inputs, to64, tol)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_forward_gb300 import build
    build.build()
    import mamba_ssd_forward_gb300 as m
    return m


@pytest.fixture(scope="module")
def O():  # noqa: E743, N802
    from oracle import layer
    return layer


# ------------------------------------------------------ causal convolution
# (b, L, D, W, wide, lengths, more)
CONV = [
    (1, 1, 8, 4, 0, None, {}),
    (2, 2, 4, 4, 0, None, {"state": False}),
    (3, 130, 260, 3, 12, [130, 0, 1], {}),
    (2, 33, 24, 2, 8, [17, 33], {"bias": False}),
    (2, 65, 33, 4, 7, None, {}),               # odd channels and an odd offset: single elements
    (1, 300, 1027, 4, 0, None, {"state": False}),
    (4, 19, 136, 4, 24, [19, 3, 2, 1], {}),    # ends within the first window
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,L,D,W,wide,lengths,more", CONV)
def test_conv(ssd, O, b, L, D, W, wide, lengths, more, dtype):
    for act in ("silu", None):
        a, gy, gfinal = conv_inputs(b, L, D, W, dtype, seed=L, wide=wide, **more)
        y, fin = ssd.causal_conv_forward(**a, lengths=lengths_of(lengths), activation=act)
        yr, fr = O.causal_conv(**host(a), lengths=lengths, act=act == "silu")
        close(y, yr, tol(y.dtype), "y")
        np.testing.assert_array_equal(to64(fin), fr)  # inputs, copied
        for gf in (gfinal, None):
            g = ssd.causal_conv_backward(**a, gy=gy, gfinal=gf, lengths=lengths_of(lengths),
                                         activation=act)
            r = O.causal_conv_backward(**host(a), gy=to64(gy), gfinal=None if gf is None else
                                       to64(gf), lengths=lengths, act=act == "silu")
            close(g["dx"], r["dx"], tol(y.dtype), "dx")
            close(g["dweight"], r["dweight"], tol(None, terms=b * L), "dweight")
            assert (g["dbias"] is None) == (a["bias"] is None)
            if a["bias"] is not None:
                close(g["dbias"], r["dbias"], tol(None, terms=b * L), "dbias")
            assert (g["dstate"] is None) == (a["state"] is None)
            if a["state"] is not None:
                close(g["dstate"], r["dstate"], tol(y.dtype), "dstate")
    ssd.device_error()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,D,W,wide", [(1, 8, 4, 0), (5, 132, 4, 4), (3, 31, 3, 5), (70, 64, 2, 0)])
def test_conv_steps_continue_the_forward(ssd, O, b, D, W, wide, dtype):
    L, cut = 9, 4
    a, _, _ = conv_inputs(b, L, D, W, dtype, seed=D, wide=wide)
    y, fin = ssd.causal_conv_forward(**a)
    y1, state = ssd.causal_conv_forward(a["x"][:, :cut], a["weight"], a["bias"], a["state"])
    assert torch.equal(y1, y[:, :cut])
    yr, _ = O.causal_conv(**host(a))
    for t in range(cut, L):
        yt = ssd.causal_conv_step(a["x"][:, t], a["weight"], a["bias"], state)
        close(yt, yr[:, t], tol(y.dtype), f"y[{t}]")
    assert torch.equal(state, fin)


# ----------------------------------------------------------- selective scan
# (b, L, D, N, G, wide, lengths, more)
SCAN = [
    (1, 1, 8, 16, 1, 0, None, {}),
    (2, 3, 5, 1, 1, 0, None, {"h0": False}),
    (3, 70, 66, 5, 3, 3, [70, 0, 1], {}),
    (2, 129, 40, 16, 1, 8, None, {"z": False}),
    (1, 257, 160, 16, 2, 0, [200], {"skip": False, "h0": False}),
    (2, 33, 12, 64, 2, 8, [32, 16], {"bias": False}),
    (1, 40, 9, 33, 1, 1, None, {}),
    (2, 300, 264, 16, 1, 24, [300, 129], {}),
]


def run_scan(O, a, gy, gfinal, lengths, softplus):
    h = host(a)
    y, fin = O.selective_scan(**h, lengths=lengths, dt_softplus=softplus)
    r = O.selective_scan_backward(**h, gy=to64(gy), gfinal=to64(gfinal), lengths=lengths,
                                  dt_softplus=softplus)
    return y, fin, r


def check_scan_grads(g, r, a, dtype, b, L, D):
    io = DTYPES[dtype]
    for k in ("du", "ddt", "dz"):
        assert (g[k] is None) == (k == "dz" and a["z"] is None)
        if g[k] is not None:
            close(g[k], r[k], tol(io, tokens=2 * L), k)
    for k in ("dB", "dC"):
        close(g[k], r[k], tol(io, tokens=2 * L, terms=D), k)
    for k, name in (("dA", "A"), ("dD", "D"), ("ddt_bias", "dt_bias")):
        assert (g[k] is None) == (a[name] is None)
        if g[k] is not None:
            close(g[k], r[k], tol(None, tokens=2 * L, terms=b * L), k)
    assert (g["dh0"] is None) == (a["h0"] is None)
    if a["h0"] is not None:
        close(g["dh0"], r["dh0"], tol(None, tokens=2 * L), "dh0")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,L,D,N,G,wide,lengths,more", SCAN)
def test_scan(ssd, O, b, L, D, N, G, wide, lengths, more, dtype):
    a, gy, gfinal = scan_inputs(b, L, D, N, G, dtype, seed=L, wide=wide, **more)
    softplus = True
    if a["dt_bias"] is None:  # without the bias: steps given as they are
        softplus = False
        a["dt"] = torch.exp(a["dt"].float() - 4.0).to(a["dt"].dtype)
    yr, fr, r = run_scan(O, a, gy, gfinal, lengths, softplus)
    y, fin = ssd.selective_scan_forward(**a, lengths=lengths_of(lengths), dt_softplus=softplus)
    close(y, yr, tol(y.dtype, tokens=L), "y")
    close(fin, fr, tol(None, tokens=L), "final_state")
    g = ssd.selective_scan_backward(**a, gy=gy, gfinal=gfinal, lengths=lengths_of(lengths),
                                    dt_softplus=softplus)
    check_scan_grads(g, r, a, dtype, b, L, D)
    ssd.device_error()


# rows on 4 bytes but not on 16
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,L,D,N,G,wide,lengths,more", [
    (2, 100, 264, 16, 1, 2, [100, 37], {}), (2, 50, 36, 14, 2, 6, None, {"h0": False}),
    (1, 21, 132, 3, 1, 1, None, {}), (2, 35, 140, 40, 1, 10, [35, 2], {"z": False}),
    (3, 18, 300, 4, 1, 0, [18, 0, 5], {"bias": False}),
])
def test_scan_rows_on_small_boundaries(ssd, O, b, L, D, N, G, wide, lengths, more, dtype):
    test_scan(ssd, O, b, L, D, N, G, wide, lengths, more, dtype)


def test_step_and_its_slope_everywhere(ssd):
    # one token and state, everything else 1: y = softplus(v), ddt = sigmoid(v)
    v = torch.linspace(-40, 40, 2001, device="cuda")
    one = torch.ones(1, 1, v.numel(), device="cuda")
    a = dict(u=one, dt=v[None, None], A=-torch.ones(v.numel(), 1, device="cuda"),
             B=one[..., :1, None], C=one[..., :1, None])
    y, _ = ssd.selective_scan_forward(**a, dt_softplus=True)
    ddt = ssd.selective_scan_backward(**a, gy=one, dt_softplus=True)["ddt"]
    w = to64(v)
    for got, ref in ((y, np.log1p(np.exp(-abs(w))) + np.maximum(w, 0)), (ddt, 1 / (1 + np.exp(-w)))):
        assert (abs(to64(got)[0, 0] - ref) <= tol(torch.float32) * ref).all()


# enough warps to cut each segment into parts; long sequences of few channels
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,L,D,N,lengths", [
    (16, 700, 640, 16, [700, 0, 1, 140, 141, 699, 560, 561, 35, 36, 420, 700, 700, 8, 9, 333]),
    (1, 3000, 8, 4, None), (2, 1500, 33, 2, [1500, 777]),
])
def test_scan_cuts(ssd, O, b, L, D, N, lengths, dtype):
    a, _, _ = scan_inputs(b, L, D, N, 1, dtype, seed=L)
    yr, fr = O.selective_scan(**host(a), lengths=lengths, dt_softplus=True)
    y, fin = ssd.selective_scan_forward(**a, lengths=lengths_of(lengths), dt_softplus=True)
    close(y, yr, tol(y.dtype, tokens=L, terms=N), "y")
    close(fin, fr, tol(torch.float32, tokens=L), "final_state")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,D,N,G,wide", [(1, 8, 16, 1, 0), (5, 130, 16, 2, 2), (3, 31, 7, 1, 5),
                                          (2, 16, 64, 1, 0)])
def test_scan_steps_continue_the_forward(ssd, O, b, D, N, G, wide, dtype):
    L, cut = 9, 4
    a, _, _ = scan_inputs(b, L, D, N, G, dtype, seed=D, wide=wide)
    yr, fr = O.selective_scan(**host(a), dt_softplus=True)
    part = {k: (v[:, :cut] if k in ("u", "dt", "B", "C", "z") else v) for k, v in a.items()}
    _, state = ssd.selective_scan_forward(**part, dt_softplus=True)
    for t in range(cut, L):
        y = ssd.selective_scan_step(*(a[k][:, t] if k in ("u", "dt", "B", "C", "z") else a[k]
                                      for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")),
                                    state, dt_softplus=True)
        close(y, yr[:, t], tol(y.dtype, tokens=L), f"y[{t}]")
    close(state, fr, tol(None, tokens=L), "state")


def test_scan_extreme_steps(ssd, O):
    """Steps so large that the decay is zero, so small that it is one, and a
    softplus far into both tails."""
    a, gy, gfinal = scan_inputs(1, 64, 16, 16, 1, "fp32", seed=4)
    dt = a["dt"]
    dt[:, ::4], dt[:, 1::4], dt[:, 2::4] = -30.0, 60.0, 4.0
    yr, fr, r = run_scan(O, a, gy, gfinal, None, True)
    y, fin = ssd.selective_scan_forward(**a, dt_softplus=True)
    close(y, yr, tol(None, tokens=64), "y")
    close(fin, fr, tol(None, tokens=64), "final_state")
    g = ssd.selective_scan_backward(**a, gy=gy, gfinal=gfinal, dt_softplus=True)
    check_scan_grads(g, r, a, "fp32", 1, 64, 16)


# -------------------------------------------------------- gated group norm
NORM = [
    (1, 8, 1, 0), (3, 12, 3, 0), (7, 33, 1, 5), (5, 66, 2, 2), (2, 1536, 1, 0), (9, 1024, 8, 8),
    (300, 320, 1, 0), (2, 5121, 1, 0), (3, 20480, 2, 0), ((2, 5), 96, 1, 16), (4, 5, 5, 0),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate,center", [("input", False), ("output", True), ("none", False),
                                         ("input", True)])
@pytest.mark.parametrize("rows,D,groups,wide", NORM)
def test_norm(ssd, O, rows, D, groups, wide, gate, center, dtype):
    a, gy = norm_inputs(rows, D, dtype, seed=D, wide=wide, gate=gate, bias=center)
    how = dict(groups=groups, gate=gate, center=center)
    h = {k: (v.reshape(-1, D) if k in ("x", "z") and v is not None else v)
         for k, v in host(a).items()}
    n = h["x"].shape[0]
    y = ssd.gated_norm_forward(**a, **how)
    assert y.shape == a["x"].shape
    close(y.reshape(n, D), O.gated_norm(**h, **how), tol(y.dtype), "y")
    g = ssd.gated_norm_backward(**a, gy=gy, **how)
    r = O.gated_norm_backward(**h, gy=to64(gy).reshape(n, D), **how)
    if D // groups > 1:
        close(g["dx"].reshape(n, D), r["dx"], tol(y.dtype), "dx")
        if gate != "none":
            close(g["dz"].reshape(n, D), r["dz"], tol(y.dtype), "dz")
    close(g["dweight"], r["dweight"], tol(None, terms=n), "dweight")
    assert (g["dbias"] is None) == (a["bias"] is None)
    if a["bias"] is not None:
        close(g["dbias"], r["dbias"], tol(None, terms=n), "dbias")
    ssd.device_error()


@pytest.mark.parametrize("D", [64, 35, 5000])
def test_norm_in_place_and_zero_rows(ssd, O, D):
    """y may be x; a row of zeros gives the bias and finite gradients."""
    a, gy = norm_inputs(6, D, "fp32", seed=1)
    a["x"][2] = 0.0
    ref = O.gated_norm(**host(a))
    h = host(a)
    g = ssd.gated_norm_backward(**a, gy=gy)
    r = O.gated_norm_backward(**h, gy=to64(gy))
    for k in ("dx", "dz"):
        # the zero row's rows are scaled by 1 / sqrt(eps): compared by themselves
        for rows in ([2], [0, 1, 3, 4, 5]):
            close(g[k][rows], r[k][rows], tol(torch.float32), k)
    out = ssd.gated_norm_forward(**a, y=a["x"])
    assert out is a["x"]
    close(out, ref, tol(torch.float32), "y in place")


# ----------------------------------------------------- norm and clipping

def test_clip(ssd, O):
    r = Draw(3)
    shapes = [(5, 7), (0,), (70001,), (1,), (3, 1, 129)] + [(k % 37 + 1,) for k in range(200)]
    base = [r.normal(*s, dtype=torch.bfloat16 if i % 3 == 0 else torch.float32)
            for i, s in enumerate(shapes)]
    flat = r.normal(1000)
    base.append(flat[3:900])  # aligned to its element only
    n = sum(t.numel() for t in base)
    for limit in (0.5, 1e5):
        grads = [t.clone() if t.numel() != 897 else t for t in base]
        ref_norm, ref = O.clip_grad_norm([to64(t) for t in grads], limit)
        out = [torch.full_like(t, float("nan")) for t in grads]
        norm = ssd.clip_grad_norm(grads, limit, out=out)
        assert norm.shape == () and norm.dtype == torch.float32
        assert abs(float(norm) - ref_norm) <= tol(None, terms=0) * ref_norm + n * 1e-12
        for o, g, t in zip(out, ref, grads):
            close(o, g, tol(t.dtype), "scaled")
            if limit == 1e5:
                assert torch.equal(o, t)  # a factor of one changes nothing
        kept = [t.clone() for t in grads]
        norm2 = ssd.clip_grad_norm(kept, limit)  # in place
        assert float(norm2) == float(norm)
        for o, k in zip(out, kept):
            assert torch.equal(o, k)
    ssd.device_error()


def test_clip_odd_values(ssd):
    """No elements; zeros; an infinity; a value that is not a number."""
    none = ssd.clip_grad_norm([torch.empty(0, device="cuda")], 1.0)
    assert float(none) == 0.0
    z = torch.zeros(100, device="cuda")
    assert float(ssd.clip_grad_norm([z], 1.0)) == 0.0 and not z.any()
    g = torch.ones(100, device="cuda")
    g[5] = float("inf")
    assert float(ssd.clip_grad_norm([g], 1.0)) == float("inf")
    assert torch.isnan(g[5]) and float(g[:5].abs().max()) == 0.0
    a, b = torch.ones(7, device="cuda"), torch.ones(3, device="cuda", dtype=torch.bfloat16)
    a[0] = float("nan")
    assert torch.isnan(ssd.clip_grad_norm([a, b], 1.0))
    assert torch.isnan(a).all() and torch.isnan(b).all()


# ------------------------------------------------- what holds for all of them

def test_padding_is_not_read(ssd):
    """Whatever stands past a sequence's end: the same results, zeros there."""
    n = [5, 0, 17]
    a, gy, gf = conv_inputs(3, 17, 24, 4, "bf16", seed=2)
    s, sgy, sgf = scan_inputs(3, 17, 24, 16, 1, "bf16", seed=2)
    lens = lengths_of(n)

    def everything(x_fill):
        out = []
        for i, k in enumerate(n):
            for t in (a["x"], gy, s["u"], s["dt"], s["B"], s["C"], s["z"], sgy):
                t[i, k:] = x_fill
        out += ssd.causal_conv_forward(**a, lengths=lens)
        g = ssd.causal_conv_backward(**a, gy=gy, gfinal=gf, lengths=lens)
        out += [g[k] for k in ("dx", "dweight", "dbias", "dstate")]
        out += ssd.selective_scan_forward(**s, lengths=lens, dt_softplus=True)
        g = ssd.selective_scan_backward(**s, gy=sgy, gfinal=sgf, lengths=lens, dt_softplus=True)
        return out + [g[k] for k in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias",
                                     "dh0")]

    clean, dirty = everything(0.0), everything(float("nan"))
    for i, (p, q) in enumerate(zip(clean, dirty)):
        assert torch.equal(p, q), i
        if p.dim() >= 3 and p.shape[1] == 17:
            for j, k in enumerate(n):
                assert not p[j, k:].any(), i


def test_lengths_out_of_range_are_clamped(ssd):
    a, _, _ = conv_inputs(2, 9, 16, 4, "fp32", seed=8)
    y, fin = ssd.causal_conv_forward(**a, lengths=lengths_of([-3, 100]))
    y2, fin2 = ssd.causal_conv_forward(**a, lengths=lengths_of([0, 9]))
    assert torch.equal(y, y2) and torch.equal(fin, fin2)


GUARD = 1024


def guarded(*shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), float("nan"), dtype=dtype, device="cuda")
    return buf, buf[GUARD:GUARD + n].view(shape)


@pytest.mark.parametrize("D", [32, 37])
def test_outputs_stay_inside_their_buffers(ssd, D):
    io, b, L, N = torch.bfloat16, 2, 21, 16
    bufs = []

    def make(*shape, dtype=io):
        buf, t = guarded(*shape, dtype=dtype)
        bufs.append((buf, t))
        return t

    a, _, _ = conv_inputs(b, L, D, 4, "bf16")
    ssd.causal_conv_forward(**a, y=make(b, L, D), final_state=make(b, 3, D))
    st = make(b, 3, D)
    st.copy_(a["state"])
    ssd.causal_conv_step(a["x"][:, 0], a["weight"], a["bias"], st, y=make(b, D))
    s, _, _ = scan_inputs(b, L, D, N, 1, "bf16")
    ssd.selective_scan_forward(**s, dt_softplus=True, y=make(b, L, D),
                               final_state=make(b, D, N, dtype=torch.float32))
    h = make(b, D, N, dtype=torch.float32)
    h.copy_(s["h0"])
    ssd.selective_scan_step(*(s[k][:, 0] if k in ("u", "dt", "B", "C", "z") else s[k] for k in
                              ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")), h,
                            dt_softplus=True, y=make(b, D))
    n, _ = norm_inputs(5, D, "bf16")
    ssd.gated_norm_forward(**n, y=make(5, D))
    g = make(3001, dtype=torch.float32)
    g.fill_(1.0)
    ssd.clip_grad_norm([g], 1.0)
    # an output that is a slice of wider rows: the columns beside it stay
    wide = torch.full((b, L, D + 8), 7.0, dtype=io, device="cuda")
    y, _ = ssd.causal_conv_forward(**a)
    ssd.causal_conv_forward(**a, y=wide[..., 3:3 + D])
    assert torch.equal(wide[..., 3:3 + D], y)
    assert bool((wide[..., :3] == 7.0).all()) and bool((wide[..., 3 + D:] == 7.0).all())
    torch.cuda.synchronize()
    for i, (buf, t) in enumerate(bufs):
        assert torch.isnan(buf[:GUARD]).all() and torch.isnan(buf[-GUARD:]).all(), i
        assert torch.isfinite(t).all(), i


def test_calls_repeat_bit_for_bit(ssd):
    a, gy, gf = conv_inputs(3, 500, 260, 4, "fp32", seed=5)
    s, sgy, sgf = scan_inputs(3, 200, 132, 16, 2, "fp32", seed=5)
    n, ngy = norm_inputs(700, 512, "fp32", seed=5)
    grads = [Draw(k).normal(40000 + k) for k in range(5)]

    def everything():
        out = list(ssd.causal_conv_backward(**a, gy=gy, gfinal=gf).values())
        out += ssd.selective_scan_forward(**s, dt_softplus=True)
        out += ssd.selective_scan_backward(**s, gy=sgy, gfinal=sgf, dt_softplus=True).values()
        out += ssd.gated_norm_backward(**n, gy=ngy).values()
        scaled = [torch.empty_like(t) for t in grads]
        return out + [ssd.clip_grad_norm(grads, 1.0, out=scaled)] + scaled

    one = everything()
    for _ in range(3):
        for i, (p, q) in enumerate(zip(one, everything())):
            assert (p is None and q is None) or torch.equal(p, q), i


def test_another_stream_and_a_graph(ssd):
    a, gy, _ = conv_inputs(2, 64, 64, 4, "bf16", seed=6)
    s, sgy, _ = scan_inputs(2, 64, 64, 16, 1, "bf16", seed=6)
    n, ngy = norm_inputs(128, 64, "bf16", seed=6)
    g = [Draw(1).normal(5000)]
    scaled = [torch.empty_like(g[0])]

    def everything():
        out = [ssd.causal_conv_forward(**a)[0], ssd.causal_conv_backward(**a, gy=gy)["dx"],
               ssd.selective_scan_forward(**s, dt_softplus=True)[0],
               ssd.selective_scan_backward(**s, gy=sgy, dt_softplus=True)["dB"],
               ssd.gated_norm_forward(**n), ssd.gated_norm_backward(**n, gy=ngy)["dweight"],
               ssd.clip_grad_norm(g, 0.5, out=scaled), scaled[0]]
        return out

    ref = [t.clone() for t in everything()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, got))


def test_offsets_beyond_31_bits(ssd, O):
    """Tokens 2^30 + 8 elements apart: the third starts past 2^31."""
    far, D, L = (1 << 30) + 8, 16, 3
    buf = torch.empty(2 * far + D, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((1, L, D), (0, far, 1))
    a, _, _ = conv_inputs(1, L, D, 4, "bf16", seed=9)
    x.copy_(a["x"])
    near, _ = ssd.causal_conv_forward(**a)
    a["x"] = x
    y, _ = ssd.causal_conv_forward(**a)
    assert torch.equal(y, near)
    a["x"] = x.contiguous()
    ssd.causal_conv_forward(**a, y=x)
    assert torch.equal(x, near)
    s, _, _ = scan_inputs(1, L, D, 16, 1, "bf16", seed=9)
    x.copy_(s["u"])
    near, _ = ssd.selective_scan_forward(**s, dt_softplus=True)
    s["u"] = x
    y, _ = ssd.selective_scan_forward(**s, dt_softplus=True)
    assert torch.equal(y, near)
    n, _ = norm_inputs(L, D, "bf16", seed=9, gate="none")
    x[0].copy_(n["x"])
    assert torch.equal(ssd.gated_norm_forward(x, n["weight"], n["bias"], gate="none"),
                       ssd.gated_norm_forward(**n, gate="none")[None])


def test_autograd_matches_the_backward_calls(ssd):
    a, gy, gf = conv_inputs(2, 20, 24, 4, "bf16", seed=12)
    s, sgy, sgf = scan_inputs(2, 20, 24, 16, 1, "bf16", seed=12)
    n, ngy = norm_inputs((2, 20), 24, "bf16", seed=12, gate="output")
    lens = lengths_of([20, 7])
    leaf = lambda d: {k: v.detach().clone().requires_grad_() for k, v in d.items()}  # noqa: E731
    la = leaf(a)
    y, fin = ssd.causal_conv(**la, lengths=lens)
    torch.autograd.backward([y, fin], [gy, gf])
    g = ssd.causal_conv_backward(**a, gy=gy, gfinal=gf, lengths=lens)
    for k in a:
        assert torch.equal(la[k].grad, g["d" + k]), k
    ls = leaf(s)
    y, fin = ssd.selective_scan(**ls, lengths=lens, dt_softplus=True)
    torch.autograd.backward([y, fin], [sgy, sgf])
    g = ssd.selective_scan_backward(**s, gy=sgy, gfinal=sgf, lengths=lens, dt_softplus=True)
    for k in s:
        assert torch.equal(ls[k].grad, g["d" + k]), k
    ln = leaf(n)
    y = ssd.gated_norm(**ln, gate="output", center=True)
    y.backward(ngy)
    g = ssd.gated_norm_backward(**n, gy=ngy, gate="output", center=True)
    for k in n:
        assert torch.equal(ln[k].grad, g["d" + k]), k
    # an expanded cotangent, as sum() sends it
    for t in la.values():
        t.grad = None
    ssd.causal_conv(**la)[0].sum().backward()
    one = ssd.causal_conv_backward(**a, gy=torch.ones_like(gy))
    assert torch.equal(la["x"].grad, one["dx"])


def test_gradients_against_differences(ssd):
    """Central differences of the kernels' own forwards, fp32: a step of 1e-2
    leaves a cubic term of 1e-4 and rounding of 1e-7 / 1e-2, so 2e-2 of the
    directional derivative's scale."""
    r = Draw(31)
    a, gy, gf = conv_inputs(2, 30, 16, 4, "fp32", seed=31)
    s, sgy, sgf = scan_inputs(2, 30, 16, 16, 1, "fp32", seed=31)
    s["B"], s["C"] = s["B"].contiguous(), s["C"].contiguous()
    n, ngy = norm_inputs(30, 16, "fp32", seed=31)

    def check(f, args, cot, grads):
        for k in args:
            v = r.normal(*args[k].shape)
            v = v / v.norm()
            vals = []
            for sgn in (1, -1):
                outs = f(**{**args, k: args[k] + sgn * 1e-2 * v})
                vals.append(sum(float((c.double() * o.double()).sum()) for c, o in zip(cot, outs)))
            diff = (vals[0] - vals[1]) / 2e-2
            want = float((grads["d" + k].double() * v.double()).sum())
            scale = float(grads["d" + k].double().norm()) / np.sqrt(v.numel())
            assert abs(diff - want) <= 2e-2 * max(abs(want), scale) + 1e-3 * scale, k

    check(lambda **k: ssd.causal_conv_forward(**k), a, (gy, gf),
          ssd.causal_conv_backward(**a, gy=gy, gfinal=gf))
    check(lambda **k: ssd.selective_scan_forward(**k, dt_softplus=True), s, (sgy, sgf),
          ssd.selective_scan_backward(**s, gy=sgy, gfinal=sgf, dt_softplus=True))
    check(lambda **k: (ssd.gated_norm_forward(**k),), n, (ngy,),
          ssd.gated_norm_backward(**n, gy=ngy))


# ------------------------------------------------------------ debug bounds

def test_debug_bounds_build(O):
    """Every operator in the build that checks its indexes: none fires."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_forward_gb300 import _abi, build
    import mamba_ssd_forward_gb300 as m
    build.build()
    release = _abi.load()
    _abi._lib = _abi.load(build.build_debug())
    try:
        for D, wide, lens in ((36, 4, [40, 9]), (33, 1, None)):
            a, gy, gf = conv_inputs(2, 40, D, 4, "bf16", wide=wide)
            y, fin = m.causal_conv_forward(**a, lengths=lengths_of(lens))
            close(y, O.causal_conv(**host(a), lengths=lens)[0], tol(y.dtype), "conv")
            m.causal_conv_backward(**a, gy=gy, gfinal=gf, lengths=lengths_of(lens))
            m.causal_conv_step(a["x"][:, 0], a["weight"], a["bias"], fin)
            s, sgy, sgf = scan_inputs(2, 40, D, 13, 3, "bf16", wide=wide)
            y, fin = m.selective_scan_forward(**s, lengths=lengths_of(lens), dt_softplus=True)
            close(y, O.selective_scan(**host(s), lengths=lens, dt_softplus=True)[0],
                  tol(y.dtype, tokens=40), "scan")
            m.selective_scan_backward(**s, gy=sgy, gfinal=sgf, lengths=lengths_of(lens),
                                      dt_softplus=True)
            m.selective_scan_step(*(s[k][:, 0] if k in ("u", "dt", "B", "C", "z") else s[k]
                                    for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")),
                                  fin, dt_softplus=True)
            n, ngy = norm_inputs(9, D, "bf16", wide=wide)
            m.gated_norm_forward(**n)
            m.gated_norm_backward(**n, gy=ngy)
            m.clip_grad_norm([Draw(2).normal(50001), Draw(2).normal(77, dtype=torch.bfloat16)],
                             1.0)
            m.device_error()
    finally:
        _abi._lib = release
