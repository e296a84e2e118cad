"""The operators around the scan at sizes where every thread has several turns
of its loops: rings of copies that come round, segments that hand over states
and adjoints, teams with several tokens, threads with several sequences, and
offsets beyond 31 bits in the gradients.  Each size is checked to be one of
those.  References in float64 (layer_ref64.py on the device, the numpy oracle
for the norm, the token and clipping); tolerances: layer_cases.py."""
import numpy as np
import pytest
import torch

import layer_ref64 as R
from layer_cases import DTYPES, close, conv_inputs, host, lengths_of, norm_inputs, scan_inputs, \
    to64, tol

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


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def near(got, ref, limit, what):
    """close() of layer_cases, on the device."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    off, norm = float((got - ref).norm()), float(ref.norm())
    assert off <= limit * norm + 1e-30, f"{what}: off by {off / max(norm, 1e-300):.3e}, " \
                                        f"limit {limit:.3e}"


# ------------------------------------------------------ causal convolution

# rows on 16 bytes, and on their element only
@pytest.mark.parametrize("wide", [0, 1])
@pytest.mark.parametrize("dtype,W,lengths,act", [
    ("bf16", 4, None, "silu"), ("bf16", 3, [8191, 5003], None), ("fp32", 2, [0, 8190], "silu"),
    ("fp32", 4, [8191, 1], "silu")])
def test_conv_of_long_runs(ssd, dtype, W, lengths, act, wide):
    b, L, D = 2, 8191, 3840 if wide == 0 else 1000
    # even with every thread that the device holds at work, each has 24 tokens
    V = (8 if dtype == "bf16" else 4) if wide == 0 else 1
    assert b * L * D / V >= 24 * sms() * 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(W)

    def normal(*shape, scale=1.0, io=DTYPES[dtype]):
        t = torch.randn(*shape[:-1], shape[-1] + wide, generator=g, device="cuda") * scale
        return t.to(io)[..., wide:]

    a = dict(x=normal(b, L, D), weight=normal(D, W, scale=0.5, io=torch.float32).contiguous(),
             bias=normal(D, scale=0.3, io=torch.float32).contiguous(),
             state=normal(b, W - 1, D).contiguous())
    n, how = lengths_of(lengths), dict(lengths=lengths, act=act == "silu")
    y, fin = ssd.causal_conv_forward(**a, lengths=n, activation=act)
    yr, fr = R.causal_conv(**a, **how)
    near(y, yr, tol(y.dtype), "y")
    assert torch.equal(fin.double(), fr)
    del y, yr
    gy, gf = normal(b, L, D), normal(b, W - 1, D).contiguous()
    need = ssd.causal_conv_backward_workspace_size(a["x"], a["weight"])
    rows = need // (4 * D * (W + 1))  # partial sums: of eight runs each
    assert b * L / (8 * rows) >= 16
    got = ssd.causal_conv_backward(**a, gy=gy, gfinal=gf, lengths=n, activation=act)
    ref = R.causal_conv_backward(**a, gy=gy, gfinal=gf, **how)
    near(got["dx"], ref["dx"], tol(a["x"].dtype), "dx")
    near(got["dstate"], ref["dstate"], tol(a["x"].dtype), "dstate")
    for k in ("dweight", "dbias"):
        near(got[k], ref[k], tol(None, terms=b * L), k)
    ssd.device_error()


# ----------------------------------------------------------- selective scan

def segments_per_part(ssd, a, cw):
    """Of the gradients, from the size of what is kept for them: states of
    every segment, adjoints of every part, partial sums of both."""
    (b, L, D), (N, G) = a["u"].shape, (a["A"].shape[1], a["B"].shape[2])
    need = ssd.selective_scan_backward_workspace_size(a["u"], a["A"], a["B"]) / 4
    tiles = -(-D // G // cw)
    ids, segs = b * G * tiles, -(-L // min(16, 512 // cw))
    parts = (need - ids * segs * (512 + cw) - 2 * tiles * b * L * G * N) / \
        (ids * (512 + cw) + b * D * (N + 2))
    return segs, round(parts), segs / round(parts)


def check_scan(ssd, a, gy, gfinal, lengths):
    b, L, D = a["u"].shape
    n, how = lengths_of(lengths), dict(lengths=lengths, dt_softplus=True)
    io = a["u"].dtype
    y, fin = ssd.selective_scan_forward(**a, lengths=n, dt_softplus=True)
    yr, fr = R.selective_scan(**a, **how)
    near(y, yr, tol(io, tokens=L), "y")
    near(fin, fr, tol(None, tokens=L), "final_state")
    got = ssd.selective_scan_backward(**a, gy=gy, gfinal=gfinal, lengths=n, dt_softplus=True)
    ref = R.selective_scan_backward(**a, gy=gy, gfinal=gfinal, **how)
    for k in ("du", "ddt", "dz"):
        near(got[k], ref[k], tol(io, tokens=2 * L), k)
    for k in ("dB", "dC"):
        near(got[k], ref[k], tol(io, tokens=2 * L, terms=D), k)
    for k in ("dA", "dD", "ddt_bias"):
        near(got[k], ref[k], tol(None, tokens=2 * L, terms=b * L), k)
    near(got["dh0"], ref["dh0"], tol(None, tokens=2 * L), "dh0")
    ssd.device_error()


# rows in pieces of 16 bytes, of 4 (bf16: wide 2), of single elements
@pytest.mark.parametrize("wide", [0, 2, 1])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,L,D,N,G,cw,lengths", [
    (16, 491, 1024, 16, 1, 32, None),
    (8, 460, 1024, 16, 2, 32, [460, 0, 1, 17, 256, 459, 33, 300]),
    (8, 250, 512, 64, 1, 8, [250, 16, 249, 0, 128, 32, 5, 250]),
    (9, 340, 1536, 8, 3, 64, None),
    (40, 300, 1500, 5, 1, 64, None),
])
def test_scan_parts_of_several_segments(ssd, b, L, D, N, G, cw, lengths, dtype, wide):
    a, gy, gfinal = scan_inputs(b, L, D, N, G, dtype, seed=L, wide=wide)
    segs, parts, per = segments_per_part(ssd, a, cw)
    assert per > 1 and 1 < parts < segs, (segs, parts)
    check_scan(ssd, a, gy, gfinal, lengths)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_scan_of_many_tokens(ssd, dtype):
    a, gy, gfinal = scan_inputs(2, 3001, 48, 16, 1, dtype, seed=1)
    check_scan(ssd, a, gy, gfinal, [3001, 2222])


# four states at a time, and one; an odd number of sequences
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,D,N,G,wide", [(31, 2816, 16, 1, 0), (65, 2560, 5, 2, 1),
                                          (21, 1024, 64, 1, 0)])
def test_token_of_several_sequences_a_thread(ssd, O, b, D, N, G, wide, dtype):
    lanes = 1 << max(0, int(np.ceil(np.log2(N / 4))))
    assert b * D * lanes >= 2 * 1024 * sms() and b % 2
    a, _, _ = scan_inputs(b, 1, D, N, G, dtype, seed=b, wide=wide)
    yr, fr = O.selective_scan(**host(a), dt_softplus=True)
    state = a.pop("h0").clone()
    y = ssd.selective_scan_step(*(a[k][:, 0] if k in ("u", "dt", "B", "C", "z") else a[k] for k in
                                  ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")), state,
                                dt_softplus=True)
    close(y, yr[:, 0], tol(y.dtype, tokens=1), "y")
    close(state, fr, tol(None, tokens=1), "state")
    ssd.device_error()


# -------------------------------------------------------- gated group norm

# vectors of 16 bytes, of two elements, of one; tokens that are whole teams'
# strides into other sequences
@pytest.mark.parametrize("wide", [0, 2, 1])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,D,groups,gate,center", [
    ((67, 301), 96, 1, "input", False), ((20300,), 224, 1, "output", True),
    ((11, 1901), 256, 2, "none", True), ((13, 401), 2048, 1, "input", True),
    ((6500,), 2024, 1, "output", False),
])
def test_norm_of_more_tokens_than_teams(ssd, O, rows, D, groups, gate, center, dtype, wide):
    # a team has a warp at least, and no more than 16 channels to a thread: even
    # with all of the device's 64 warps an SM at work, each has two tokens
    n, warps = int(np.prod(rows)), max(1, D // groups // 512)
    assert n * groups >= 2 * 64 * sms() / warps
    a, gy = norm_inputs(rows, D, dtype, seed=D, wide=wide, gate=gate, bias=center)
    how = dict(groups=groups, gate=gate, center=center)
    h = {k: (v.reshape(-1, D) if k in ("x", "z") and v is not None else v)
         for k, v in host(a).items()}
    y = ssd.gated_norm_forward(**a, **how)
    close(y.reshape(n, D), O.gated_norm(**h, **how), tol(y.dtype), "y")
    g = ssd.gated_norm_backward(**a, gy=gy, **how)
    r = O.gated_norm_backward(**h, gy=to64(gy).reshape(n, D), **how)
    close(g["dx"].reshape(n, D), r["dx"], tol(y.dtype), "dx")
    if gate != "none":
        close(g["dz"].reshape(n, D), r["dz"], tol(y.dtype), "dz")
    close(g["dweight"], r["dweight"], tol(None, terms=n), "dweight")
    if center:
        close(g["dbias"], r["dbias"], tol(None, terms=n), "dbias")
    ssd.device_error()


# ----------------------------------------------------- norm and clipping

def test_clip_of_many_chunks(ssd, O):
    """More pieces than blocks in one launch, in both types, on 16 bytes and off."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    flat = torch.randn(12_000_007, generator=g, device="cuda")
    grads = [flat[:7_000_001], flat[7_000_002:], flat[:9_000_000].bfloat16(),
             flat[:4_000_001].bfloat16()[1:]]
    assert sum(t.numel() * t.element_size() for t in grads) / 131072 >= 3 * sms()
    ref_norm, ref = O.clip_grad_norm([to64(t) for t in grads], 2.0)
    out = [torch.empty_like(t) for t in grads]
    norm = ssd.clip_grad_norm(grads, 2.0, out=out)
    # the sum over 512 threads of 456 blocks has chains of 200 additions at most
    assert abs(float(norm) - ref_norm) <= tol(None, terms=200) * ref_norm
    for o, r, t in zip(out, ref, grads):
        close(o, r, tol(t.dtype, terms=200), "scaled")
    ssd.device_error()


# ------------------------------------------------------ offsets past 31 bits

def far_apart(t, far):
    """The tokens of t [1, L, D], each `far` elements behind the one before."""
    _, L, D = t.shape
    buf = torch.empty((L - 1) * far + D, dtype=t.dtype, device="cuda")
    v = buf.as_strided((1, L, D), (0, far, 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("odd", [0, 1])
def test_gradients_beyond_31_bits(ssd, odd):
    """Tokens 2^30 + 8 elements apart (or 2^30 + 9): the third starts past 2^31."""
    far, L, D = (1 << 30) + 8 + odd, 3, 16
    a, gy, gf = conv_inputs(1, L, D, 4, "bf16", seed=9)
    s, sgy, sgf = scan_inputs(1, L, D, 16, 1, "bf16", seed=9)
    n, ngy = norm_inputs((1, L), D, "bf16", seed=9)
    for fn, args, names in (
            (ssd.causal_conv_backward, dict(a, gy=gy, gfinal=gf), ("x", "gy")),
            (ssd.selective_scan_backward, dict(s, gy=sgy, gfinal=sgf, dt_softplus=True),
             ("u", "dt", "z", "gy")),
            (ssd.gated_norm_backward, dict(n, gy=ngy), ("x", "z", "gy"))):
        near_by = fn(**args)
        for k in names:
            got = fn(**{**args, k: far_apart(args[k], far)})
            for g, r in near_by.items():
                if odd:  # single elements: sums in another order
                    near(got[g], r.double(), tol(r.dtype, tokens=2 * L, terms=L), (k, g))
                else:
                    assert torch.equal(got[g], r), (k, g)
    ssd.device_error()


def test_gradients_stored_beyond_31_bits(ssd):
    """dx, du, ddt, dz and dB as views whose third token starts past 2^31."""
    from mamba_ssd_forward_gb300 import _abi
    from mamba_ssd_forward_gb300.layer import _scan_inputs, _scan_dims
    lib, io = _abi.load(), torch.bfloat16
    far, L, D, N = (1 << 30) + 8, 3, 16, 16
    buf = torch.empty(2 * far + D, dtype=io, device="cuda")
    at = _abi.SsdSeq(buf.data_ptr(), 0, far)
    stored = buf.as_strided((1, L, D), (0, far, 1))
    stream = torch.cuda.current_stream().cuda_stream

    def seq(t):
        return _abi.SsdSeq(t.data_ptr(), 0, t.stride(1))

    a, gy, _ = conv_inputs(1, L, D, 4, "bf16", seed=9)
    ref = ssd.causal_conv_backward(**a, gy=gy)
    ws = torch.empty(ssd.causal_conv_backward_workspace_size(a["x"], a["weight"]),
                     dtype=torch.uint8, device="cuda")
    _abi.check("conv", lib.ssd_causal_conv_backward(
        _abi.SsdConvDims(1, L, D, 4, 1), _abi.SSD_BF16, seq(a["x"]), a["weight"].data_ptr(),
        a["bias"].data_ptr(), a["state"].data_ptr(), seq(gy), None, None, at, None, None, None,
        ws.data_ptr(), ws.numel(), stream))
    assert torch.equal(stored, ref["dx"])
    n, ngy = norm_inputs((1, L), D, "bf16", seed=9)
    ref = ssd.gated_norm_backward(**n, gy=ngy)
    ws = torch.empty(ssd.gated_norm_backward_workspace_size(n["x"]), dtype=torch.uint8,
                     device="cuda")
    dense = torch.empty_like(n["x"])
    for dx, dz, k in ((at, seq(dense), "dx"), (seq(dense), at, "dz")):
        _abi.check("norm", lib.ssd_gated_norm_backward(
            _abi.SsdNormDims(1, L, D, 1, 1e-5, _abi.SSD_GATE_INPUT, 0), _abi.SSD_BF16,
            seq(n["x"]), n["weight"].data_ptr(), n["bias"].data_ptr(), seq(n["z"]), seq(ngy), dx,
            dz, None, None, ws.data_ptr(), ws.numel(), stream))
        assert torch.equal(stored, ref[k])
    s, sgy, _ = scan_inputs(1, L, D, N, 1, "bf16", seed=9)
    ref = ssd.selective_scan_backward(**s, gy=sgy, dt_softplus=True)
    ws = torch.empty(ssd.selective_scan_backward_workspace_size(s["u"], s["A"], s["B"]),
                     dtype=torch.uint8, device="cuda")
    d = _scan_dims(s["u"], s["A"], s["B"], True)
    args = _scan_inputs(d, *(s[k] for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")))
    for k in ("du", "ddt", "dz", "dB", "dC"):
        own = {j: torch.empty(1, L, D, dtype=io, device="cuda")
               for j in ("du", "ddt", "dz", "dB", "dC")}
        g = _abi.SsdScanGrads(**{j: at if j == k else seq(t) for j, t in own.items()})
        _abi.check("scan", lib.ssd_selective_scan_backward(
            *args, s["h0"].data_ptr(), seq(sgy), None, None, g, ws.data_ptr(), ws.numel(),
            stream))
        assert torch.equal(stored, ref[k].view(1, L, D)), k
    ssd.device_error()


# ------------------------------------------------------------ debug bounds

def test_debug_bounds_build(ssd, O):
    """The same loops in the build that checks its indexes: none fires."""
    from mamba_ssd_forward_gb300 import _abi, build
    release = _abi.load()
    _abi._lib = _abi.load(build.build_debug())
    try:
        for wide in (0, 1):
            test_conv_of_long_runs(ssd, "bf16", 4, [8191, 5003], "silu", wide)
            for case in ((16, 491, 1024, 16, 1, 32, None),
                         (8, 250, 512, 64, 1, 8, [250, 16, 249, 0, 128, 32, 5, 250])):
                test_scan_parts_of_several_segments(ssd, *case, "bf16", wide)
            test_token_of_several_sequences_a_thread(ssd, O, 65, 2560, 5, 2, wide, "bf16")
            for case in (((67, 301), 96, 1, "input", False), ((13, 401), 2048, 1, "input", True)):
                test_norm_of_more_tokens_than_teams(ssd, O, *case, "bf16", wide)
        test_clip_of_many_chunks(ssd, O)
    finally:
        _abi._lib = release
