"""The operators around a language model's blocks on the GPU against their float64
definitions: small and odd sizes, types, strides, tokens without a target, and the
values at which they can go wrong.  Bounds: tests/model_ref64.py."""
import math

import pytest
import torch

import model_ref64 as R

pytestmark = pytest.mark.gpu

B16, F32 = torch.bfloat16, torch.float32
IO = {"bf16": B16, "fp32": F32}


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_forward_gb300 import build
    build.build()
    import mamba_ssd_forward_gb300 as m
    yield m
    from mamba_ssd_forward_gb300 import _abi
    assert _abi.load().ssd_device_error(torch.cuda.current_stream().cuda_stream) == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, scale=1.0, dtype=F32: \
        (torch.randn(s, generator=g, device="cuda") * scale).to(dtype)


def within(got, ref, bound, what=""):
    got, ref = got.double(), ref.double()
    off = (got - ref).abs()
    assert got.shape == ref.shape, what
    worst = (off - bound).max()
    assert not bool(torch.isnan(off).any()) and float(worst) <= 0, \
        f"{what}: off by {float(off.max()):.3e}, over the bound by {float(worst):.3e}"


def view(t, kind):
    """The same values as they are, in a slice of wider rows, or off the 16-byte grid."""
    if kind == "dense":
        return t
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + (16 if kind == "slice" else 3),
                       dtype=t.dtype, device=t.device)
    at = 8 if kind == "slice" else 1
    wide[..., at:at + t.shape[-1]] = t
    return wide[..., at:at + t.shape[-1]]


# ------------------------------------------------------ residual and norm

NORM_SHAPES = [(1, 1), (3, 2), (5, 64), (9, 257), (33, 771), (1000, 256), (7, 2560), (4, 5123),
               (700, 1003), (5, 8192), (2, 16384), (3, 16383)]
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]


@pytest.mark.parametrize("io,stream", TYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_add_norm(ssd, shape, io, stream):
    n, D = gen(sum(shape)), shape[1]
    x, r = n(*shape, dtype=IO[io]), n(*shape, scale=2.0, dtype=IO[stream])
    w = 1.0 + n(D, scale=0.2)
    y, total = ssd.add_norm_forward(x, r, w)
    ref, t = R.add_norm(x, r, w)
    within(y, ref, ref.abs() * R.norm_bound(D, IO[io]) + 2.0 ** -24 * w.double().abs(), "y")
    within(total, t, t.abs() * R.HALF[IO[stream]], "total")
    gy, gt = n(*shape, dtype=IO[io]), n(*shape, dtype=IO[stream])
    for gtotal in (gt, None):
        g = ssd.add_norm_backward(total, w, gy, gtotal)
        dt, dw = R.add_norm_backward(total, w, gy, gtotal)
        # dt = r (g w - n m) + gt: each part by the norm's bound of its own size
        tt = total.double()
        rstd = ((tt ** 2).mean(-1, keepdim=True) + 1e-5) ** -0.5
        gw = gy.double() * w.double()
        m = (gw.abs() * tt.abs()).mean(-1, keepdim=True) * rstd
        parts = rstd * (gw.abs() + tt.abs() * rstd * m) + (0 if gtotal is None else gt.double().abs())
        off = parts * (D + 16) * 2.0 ** -24
        within(g["dx"], dt, off + dt.abs() * R.HALF[IO[io]], "dx")
        within(g["dresidual"], dt, off + dt.abs() * R.HALF[IO[stream]], "dresidual")
        terms = (gy.double() * tt * rstd).abs().sum(0)
        within(g["dweight"], dw, terms * (shape[0] + D / 2 + 16) * 2.0 ** -24, "dweight")


@pytest.mark.parametrize("block", [0, 32, 64, 128])
@pytest.mark.parametrize("io,stream", TYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_add_norm_quantized(ssd, shape, io, stream, block):
    n, D = gen(sum(shape) + block), shape[1]
    x, r = n(*shape, dtype=IO[io]), n(*shape, scale=2.0, dtype=IO[stream])
    w = 1.0 + n(D, scale=0.2)
    q, scales, total = ssd.add_norm_quantized(x, r, w, block=block)
    ref, t = R.add_norm(x, r, w)
    c = block or D
    assert q.dtype == torch.float8_e4m3fn and scales.shape == (shape[0], -(-D // c))
    near = R.norm_bound(D, F32) + 2.0 ** -21
    for i, part in enumerate(ref.split(c, 1)):
        top = part.abs().amax(1)
        within(scales[:, i], top / 448, top / 448 * near, "scale")
        back = q[:, i * c:i * c + part.shape[1]].double() * scales[:, i:i + 1].double()
        # half a step of e4m3, which below 2^-6 are 2^-9 apart
        within(back, part, part.abs() * (R.HALF[q.dtype] * (1 + near) + near)
               + scales[:, i:i + 1].double() * 2.0 ** -10, "value")
        assert (back.abs().amax(1) >= top * (1 - 2 * near)).all()  # the largest is 448
    within(total, t, t.abs() * R.HALF[IO[stream]], "total")


@pytest.mark.parametrize("kind", ["slice", "off"])
@pytest.mark.parametrize("D", [96, 2560])
def test_add_norm_views_and_sequences(ssd, D, kind):
    """[b, L, D] views give the bits that dense tensors give, but for the order of the
    sums off the 16-byte grid."""
    n = gen(D)
    x, r, w = n(3, 11, D, dtype=B16), n(3, 11, D), 1.0 + n(D, scale=0.2)
    gy, gt = n(3, 11, D, dtype=B16), n(3, 11, D)
    y, total = ssd.add_norm_forward(x, r, w)
    yv, tv = ssd.add_norm_forward(view(x, kind), view(r, kind), w,
                                  y=view(torch.zeros_like(x), kind),
                                  total=view(torch.zeros_like(r), kind))
    assert torch.equal(total, tv)
    within(yv, y, y.double().abs() * 2 * R.norm_bound(D, B16) + 1e-6)
    g = ssd.add_norm_backward(total, w, gy, gt)
    gv = ssd.add_norm_backward(view(total, kind), w, view(gy, kind), view(gt, kind))
    for k in g:
        within(gv[k], g[k], g[k].double().abs() * 2 * R.HALF[g[k].dtype] + (D + 40) * 2.0 ** -22, k)
    q, s, _ = ssd.add_norm_quantized(view(x, kind), view(r, kind), w, block=64)
    q0, s0, _ = ssd.add_norm_quantized(x, r, w, block=64)
    within(s, s0, s0.double() * 2.0 ** -20)
    assert float((q.float() != q0.float()).double().mean()) < 1e-3


def test_add_norm_in_place_and_without_a_residual(ssd):
    n = gen(3)
    x, r, w = n(50, 640, dtype=B16), n(50, 640), 1.0 + n(640, scale=0.2)
    y, total = ssd.add_norm_forward(x, r, w)
    a, b = x.clone(), r.clone()
    ya, tb = ssd.add_norm_forward(a, b, w, y=a, total=b)
    assert ya is a and tb is b and torch.equal(a, y) and torch.equal(b, total)
    y0, t0 = ssd.add_norm_forward(x, None, w)
    assert t0 is None
    y1, t1 = ssd.add_norm_forward(x, None, w, total=torch.empty_like(r))
    assert torch.equal(y0, y1) and torch.equal(t1, x.float())
    ref, _ = R.add_norm(x, None, w)
    within(y0, ref, ref.abs() * R.norm_bound(640, B16) + 1e-7)
    q, s, t = ssd.add_norm_quantized(x, None, w)
    assert t is None and q.shape == x.shape


def test_add_norm_values_at_the_ends(ssd):
    """A row's infinity or NaN stays its own; rows of zeros have scale zero; scales do not
    fall below 2^-126."""
    x = torch.zeros(6, 256, device="cuda")
    x[1, 7], x[2, 9], x[3] = math.inf, math.nan, 1e-30
    x[4], x[5] = 1.0, torch.arange(256, device="cuda") * 1e-3
    r, w = torch.zeros_like(x), torch.ones(256, device="cuda")
    y, total = ssd.add_norm_forward(x, r, w)
    assert torch.equal(torch.isfinite(y).all(1).cpu(),
                       torch.tensor([True, False, False, True, True, True]))
    assert (y[0] == 0).all() and torch.equal(total[[0, 3, 4, 5]], x[[0, 3, 4, 5]])
    q, s, _ = ssd.add_norm_quantized(x, r, w, block=128)
    assert (s[0] == 0).all() and (q[0].float() == 0).all()
    assert torch.isnan(q[2].float()).all()
    tiny = torch.full((256,), 1e-39, device="cuda")
    q, s, _ = ssd.add_norm_quantized(x, r, tiny, block=0)
    assert float(s[4]) == 2.0 ** -126
    within(q[4].double() * s[4].double(), torch.full((256,), 1e-39, dtype=torch.float64,
                                                      device="cuda"), 1e-39 / 16 + 2.0 ** -136)
    huge = torch.full((256,), 1e38, device="cuda")  # a scale whose block is near the range's end
    for block in (0, 64):
        q, s, _ = ssd.add_norm_quantized(x, r, huge, block=block)
        ref, _ = R.add_norm(x[5:], r[5:], huge)
        near = R.norm_bound(256, F32) + 2.0 ** -21
        step = s[5:].double().repeat_interleave(256 // s.shape[1], 1)
        within(q[5:].double() * step, ref,
               ref.abs() * (R.HALF[q.dtype] * (1 + near) + near) + step * 2.0 ** -10, "huge")


def test_offsets_beyond_32_bits(ssd):
    """Rows so far apart that their places pass 2^32 elements: the bits of dense ones."""
    base, n = torch.empty(2 ** 32 + 2 ** 20, dtype=B16, device="cuda"), gen(31)

    def far(t, at):
        """t's rows spread over `base`, from element `at` on."""
        v = base.as_strided(t.shape, (2 ** 32 // (t.shape[0] - 1) // 8 * 8, *t.stride()[1:]), at)
        return v.copy_(t)

    x, r, w = n(2, 5, 640, dtype=B16), n(2, 5, 640, dtype=B16), 1.0 + n(640, scale=0.2)
    y, total = ssd.add_norm_forward(x, r, w)
    yv, tv = far(y, 0).zero_(), far(y, 65536).zero_()
    ssd.add_norm_forward(far(x, 131072), far(r, 262144), w, y=yv, total=tv)
    assert torch.equal(yv, y) and torch.equal(tv, total)
    g = ssd.add_norm_backward(total, w, x, r)
    v = ssd.add_norm_backward(tv, w, far(x, 131072), far(r, 262144))
    assert all(torch.equal(g[k], v[k]) for k in g)

    W, t = n(9, 640, dtype=B16), torch.tensor([[0, 8, 3, 1, -100], [8, 7, 2, 5, 6]], device="cuda")
    ref = ssd.linear_cross_entropy_forward(x, W, t)
    for at in (0, 1):  # taken where they lie, and packed
        words = far(W, at)
        got = ssd.linear_cross_entropy_forward(far(x, 524288), words, t)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
        g = ssd.linear_cross_entropy_backward(x, W, t, ref[1])
        v = ssd.linear_cross_entropy_backward(far(x, 524288), words, t, ref[1])
        assert all(torch.equal(g[k], v[k]) for k in g)

    G = n(2, 64, 128, dtype=B16)
    X = ssd.orthogonalize(G)
    out = far(X, 0).zero_()
    ssd.orthogonalize(far(G, 65536), out=out)
    assert torch.equal(out, X)


# ---------------------------------------------------------- cross entropy

LOSS_SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 7), (5, 64, 257), (130, 72, 1000), (257, 100, 513),
               (64, 2560, 300), (600, 33, 3001), (16, 40, 60000)]
IGNORED = {"none": 0.0, "some": 0.4, "all": 1.0}


def loss_case(shape, io, ignored, seed=0):
    rows, d, V = shape
    n = gen(rows + d + V + seed)
    x, w = n(rows, d, dtype=IO[io]), n(V, d, scale=2.0 / math.sqrt(d), dtype=IO[io])
    t = torch.randint(0, V, (rows,), device="cuda")
    t[torch.rand(rows, device="cuda") < IGNORED[ignored]] = -100
    if ignored == "some":
        t[0], t[-1] = -100, V - 1
    return x, w, t, n


def check_loss(ssd, x, w, t, g, io, d, V):
    ref, ref_lse, live = R.cross_entropy(x, w, t)
    z = R.logit_bound(x, w, IO[io], live)
    loss, lse = ssd.linear_cross_entropy_forward(x, w, t)
    shape, rows = t.shape, int(t.numel())
    within(loss.reshape(-1), ref, R.loss_bound(z, V, ref), "loss")
    within(lse.reshape(-1), ref_lse, R.loss_bound(z, V, ref_lse), "lse")
    assert loss.shape == lse.shape == shape
    top = float(ref_lse.abs().max())
    scale = 1.0 / max(1, int(live.sum()))
    for reduction, factor in (("none", g), ("sum", torch.full_like(g, 0.75)),
                              ("mean", torch.full_like(g, 0.75 * scale))):
        if reduction != "none":
            total, again = ssd.linear_cross_entropy_forward(x, w, t, reduction=reduction)
            assert torch.equal(lse, again)
            s = ref.sum() * (scale if reduction == "mean" else 1.0)
            each = float(R.loss_bound(z, V, ref).sum()) + rows * 2.0 ** -24 * float(ref.abs().sum())
            within(total, s, each * (scale if reduction == "mean" else 1.0) + 1e-30, reduction)
        gl = g if reduction == "none" else torch.tensor(0.75, device="cuda")
        r = ssd.linear_cross_entropy_backward(x, w, t, lse, gl, reduction=reduction)
        dx, dw, ax, aw = R.cross_entropy_backward(x, w, t, factor)
        within(r["dx"], dx, R.grad_bound(z, top, ax, V, dx, IO[io]), f"dx {reduction}")
        within(r["dweight"], dw, R.grad_bound(z, top, aw, rows, dw, IO[io]),
               f"dweight {reduction}")
        assert (r["dx"].reshape(rows, d)[~live] == 0).all()
    none = ssd.linear_cross_entropy_backward(x, w, t, lse)  # gloss 1
    ones = ssd.linear_cross_entropy_backward(x, w, t, lse, torch.ones_like(g))
    for k in none:
        dx, dw, ax, aw = R.cross_entropy_backward(x, w, t, torch.ones_like(g))
        a, b = (dx, ax) if k == "dx" else (dw, aw)
        for got in (none, ones):
            within(got[k], a, R.grad_bound(z, top, b, V if k == "dx" else rows, a, IO[io]), k)


@pytest.mark.parametrize("ignored", list(IGNORED))
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", LOSS_SHAPES, ids=str)
def test_linear_cross_entropy(ssd, shape, io, ignored):
    x, w, t, n = loss_case(shape, io, ignored)
    check_loss(ssd, x, w, t, n(shape[0]), io, shape[1], shape[2])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["slice", "off"])
def test_linear_cross_entropy_views(ssd, kind, io):
    """[b, L, D] slices of wider rows, and a vocabulary that is a slice itself."""
    n = gen(5)
    x = view(n(3, 50, 64, dtype=IO[io]), kind)
    w = view(n(500, 64, scale=0.3, dtype=IO[io]), kind)
    t = torch.randint(0, 500, (3, 50), device="cuda")
    t[1, 20:] = -100
    check_loss(ssd, x, w, t, n(3, 50), io, 64, 500)


@pytest.mark.parametrize("io,shape", [("bf16", (66000, 16, 5000)), ("fp32", (33000, 24, 4500))])
def test_linear_cross_entropy_in_pieces(ssd, io, shape):
    """So many tokens that the gradients take the vocabulary in several pieces."""
    x, w, t, n = loss_case(shape, io, "some")
    check_loss(ssd, x, w, t, n(shape[0]), io, shape[1], shape[2])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_left_out_rows_reach_nothing(ssd, io):
    """Infinities and NaN in tokens without a target."""
    x, w, t, n = loss_case((200, 48, 700), io, "some")
    g = n(200)
    lse = ssd.linear_cross_entropy_forward(x, w, t)[1]
    ref = ssd.linear_cross_entropy_backward(x, w, t, lse, g)
    dead = torch.nonzero(t == -100).flatten()
    y, h = x.clone(), g.clone()
    y[dead[::2]], y[dead[1::2]] = math.nan, math.inf
    h[dead] = math.nan
    loss, lse2 = ssd.linear_cross_entropy_forward(y, w, t)
    assert torch.equal(lse, lse2) and torch.isfinite(loss).all()
    got = ssd.linear_cross_entropy_backward(y, w, t, lse2, h)
    for k in got:
        assert torch.equal(got[k], ref[k]), k
    # nor does what lies in the workspace
    need = ssd.linear_cross_entropy_backward_workspace_size(y, w)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    got = ssd.linear_cross_entropy_backward(y, w, t, lse2, h, workspace=ws)
    for k in got:
        assert torch.equal(got[k], ref[k]), k


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_targets_that_are_no_words(ssd, io):
    x, w, t, n = loss_case((40, 32, 100), io, "none")
    t[3], t[4], t[5] = 100, -1, 1 << 40
    loss, lse = ssd.linear_cross_entropy_forward(x, w, t)
    assert torch.isnan(loss[3:6]).all() and torch.isfinite(loss[:3]).all()
    assert torch.isfinite(loss[6:]).all() and torch.isfinite(lse).all()
    r = ssd.linear_cross_entropy_backward(x, w, t, lse)
    assert torch.isnan(r["dx"][3:6]).all() and torch.isfinite(r["dx"][6:]).all()
    assert torch.isnan(r["dweight"]).all()
    # another number may stand for none: -1 as the ignored one, and -100 as no word
    t[3], t[5] = 0, 7
    loss, _ = ssd.linear_cross_entropy_forward(x, w, t, ignore_index=-1)
    assert float(loss[4]) == 0 and torch.isfinite(loss).all()


def test_logits_at_the_ends(ssd):
    """Rows with NaN or infinite logits are theirs alone; logits of the type's lowest
    value and spread over its range leave finite losses."""
    x = torch.zeros(5, 16, dtype=B16, device="cuda")
    w = torch.zeros(300, 16, dtype=B16, device="cuda")
    w[:, 0] = torch.linspace(-1, 1, 300, device="cuda")
    w[299, 0] = 1
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 1e4, math.inf, math.nan, -torch.finfo(B16).max
    t = torch.full((5,), 299, device="cuda")
    t[3] = 0
    loss, lse = ssd.linear_cross_entropy_forward(x, w, t)
    assert torch.isfinite(loss[[0, 3, 4]]).all() and torch.isnan(loss[2])
    assert not torch.isfinite(loss[1])
    within(loss[4:], torch.tensor([math.log(300)], device="cuda"), 1e-5)
    assert abs(float(loss[0])) < 1e-3 * 1e4 and abs(float(loss[3])) < 1e-5
    dx = ssd.linear_cross_entropy_backward(x, w, t, lse, want=("dx",))
    assert dx["dweight"] is None and torch.isfinite(dx["dx"][[0, 3, 4]]).all()


def test_an_infinite_fp32_row_costs_the_others_nothing(ssd):
    x, w, t, n = loss_case((70, 64, 300), "fp32", "none")
    x *= 2.0 ** 20
    w *= 2.0 ** -20
    lse = ssd.linear_cross_entropy_forward(x, w, t)[1]
    y, keep = x.clone(), torch.arange(70, device="cuda") != 9
    y[9, 3] = math.inf
    loss, got = ssd.linear_cross_entropy_forward(y, w, t)
    assert not torch.isfinite(loss[9]) and torch.equal(got[keep], lse[keep])
    dx = ssd.linear_cross_entropy_backward(y, w, t, got, want=("dx",))["dx"]
    ref = ssd.linear_cross_entropy_backward(x, w, t, lse, want=("dx",))["dx"]
    assert torch.equal(dx[keep], ref[keep])


@pytest.mark.parametrize("tokens", [8192, 8193, 20000])
def test_many_tokens_with_few_targets(ssd, tokens):
    """Targets counted by the packing blocks themselves, and in groups."""
    n = gen(tokens)
    x, w = n(tokens, 24, dtype=B16), n(90, 24, scale=0.4, dtype=B16)
    t = torch.full((tokens,), -100, device="cuda")
    t[::97] = torch.arange(len(t[::97]), device="cuda") % 90
    t[-1] = 5
    check_loss(ssd, x, w, t, n(tokens), "bf16", 24, 90)


@pytest.mark.parametrize("size", [1e-25, 1e-6, 1e6, 1e15])
def test_fp32_operands_of_any_size(ssd, size):
    """x and W scaled against one another: the same logits."""
    x, w, t, n = loss_case((70, 64, 300), "fp32", "none")
    a, b = x * 2.0 ** round(math.log2(size)), w * 2.0 ** -round(math.log2(size))
    lse = ssd.linear_cross_entropy_forward(x, w, t)[1]
    loss, got = ssd.linear_cross_entropy_forward(a, b, t)
    assert torch.equal(lse, got)
    g = n(70) * 1e-12
    r = ssd.linear_cross_entropy_backward(a, b, t, got, g)
    s = ssd.linear_cross_entropy_backward(x, w, t, got, g)
    k = 2.0 ** round(math.log2(size))
    assert torch.equal(r["dx"], s["dx"] / k) and torch.equal(r["dweight"], s["dweight"] * k)


# ---------------------------------------------------------- orthogonalisation

ORTH_SHAPES = [(1, 1), (1, 40), (50, 1), (16, 16), (77, 333), (333, 77), (256, 512), (512, 256),
               (300, 1100), (700, 700), (1030, 260), (3, 64, 129), (4, 257, 31), (2, 520, 520),
               # long and narrow: the smaller Gram matrix in parts
               (40, 3000), (5000, 1), (3, 2777, 70), (2, 300, 2500), (400, 6000)]


def relative(got, ref):
    off = (got.double() - ref).reshape(-1, *ref.shape[-2:])
    return float((torch.linalg.matrix_norm(off)
                  / torch.linalg.matrix_norm(ref.reshape(off.shape))).max())


@pytest.mark.parametrize("to", ["bf16", "fp32"])
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", ORTH_SHAPES, ids=str)
def test_orthogonalize(ssd, shape, io, to):
    G = gen(sum(shape))(*shape, scale=1e-3, dtype=IO[io])
    X = ssd.orthogonalize(G, dtype=IO[to])
    assert X.dtype == IO[to] and X.shape == G.shape
    assert relative(X, R.orthogonalize(G)) <= R.orth_bound(IO[to], G)


@pytest.mark.parametrize("to", ["bf16", "fp32"])
@pytest.mark.parametrize("steps", [1, 2, 3, 7])
def test_orthogonalize_steps_and_coefficients(ssd, steps, to):
    G = gen(steps)(90, 200)
    c = (1.875, -1.25, 0.375)
    X = ssd.orthogonalize(G, steps=steps, coefficients=c, dtype=IO[to])
    assert relative(X, R.orthogonalize(G, steps, c)) <= R.orth_bound(IO[to], G, steps, c)


@pytest.mark.parametrize("to", ["bf16", "fp32"])
def test_orthogonalize_of_few_directions(ssd, to):
    """Two strong directions over a floor of noise 2000 times smaller."""
    n = gen(9)
    G = (n(128, 2) @ n(2, 192) + 5e-4 * n(128, 192)).to(B16)
    assert relative(ssd.orthogonalize(G, dtype=IO[to]), R.orthogonalize(G)) <= R.orth_bound(IO[to], G)


@pytest.mark.parametrize("kind", ["slice", "off"])
def test_orthogonalize_views(ssd, kind):
    n = gen(4)
    for to in (B16, F32):
        G = n(2, 100, 72, dtype=B16)
        X = ssd.orthogonalize(G, dtype=to)
        out = view(torch.zeros(2, 100, 72, dtype=to, device="cuda"), kind)
        got = ssd.orthogonalize(view(G, kind), out=out)
        assert got is out
        # (another order of the norm's sums)
        assert relative(got, X.double()) <= R.HALF[to] * 2 + 2.0 ** -18
        base = out._base
        assert float(base.double().abs().sum()) == float(out.double().abs().sum())
    H = n(100, 72, dtype=B16)
    ref = ssd.orthogonalize(H)
    assert ssd.orthogonalize(H, out=H) is H and torch.equal(H, ref)


def test_orthogonalize_values_at_the_ends(ssd):
    """Zeros stay zeros, a NaN or an infinity spoils its own matrix only, sizes cancel."""
    n = gen(6)
    G = n(4, 64, 96)
    G[1] = 0
    G[2, 3, 4] = math.nan
    for to in (B16, F32):
        X = ssd.orthogonalize(G, dtype=to)
        assert (X[1] == 0).all() and torch.isnan(X[2]).any()
        for i in (0, 3):
            assert torch.equal(X[i], ssd.orthogonalize(G[i], dtype=to))
        for k in (2.0 ** -30, 2.0 ** 40):  # above eps the norm divides exactly
            Y = ssd.orthogonalize(G[:1] * k, eps=1e-30, dtype=to)
            assert torch.equal(Y, ssd.orthogonalize(G[:1], eps=1e-30, dtype=to))
        inf = G[:1].clone()
        inf[0, 0, 0] = math.inf
        assert not torch.isfinite(ssd.orthogonalize(inf, dtype=to)).all()
