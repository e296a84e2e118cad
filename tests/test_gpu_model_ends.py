"""The operators around a language model's blocks where their types, panes and number
ranges end, on the GPU against their float64 definitions.  Bounds: tests/model_ref64.py."""
import pytest
import torch

import model_ref64 as R
from test_gpu_model import (B16, F32, IO, check_loss, gen, loss_case, relative, ssd,  # noqa: F401
                            within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------- cross entropy

@pytest.mark.parametrize("io,shape", [("bf16", (66000, 20, 5000)), ("fp32", (33000, 27, 4500)),
                                      ("bf16", (300, 333, 1500)), ("fp32", (300, 771, 1500))])
def test_dweight_off_the_grid_behind_dx_tiles(ssd, io, shape):  # noqa: F811
    """Rows of dW that no bulk copy can write, whose warps come from tiles of dx with
    stores still on their way: in one piece of the vocabulary, and in several, which
    add to dx."""
    x, w, t, n = loss_case(shape, io, "some")
    check_loss(ssd, x, w, t, n(shape[0]), io, shape[1], shape[2])


@pytest.mark.parametrize("ex,ew", [(-60, -60), (-30, -75), (-110, 5)])
@pytest.mark.parametrize("V", [300, 320])
def test_fp32_logits_that_vanish(ssd, V, ex, ew):  # noqa: F811
    """x and W so small that no fp32 holds the power of two that takes the products of
    their planes to logits: a loss of log V, with and without words that fill up a tile."""
    x, w, t, n = loss_case((70, 64, V), "fp32", "some")
    check_loss(ssd, x * 2.0 ** ex, w * 2.0 ** ew, t, n(70), "fp32", 64, V)


@pytest.mark.parametrize("shape", [(130, 64, 300), (300, 77, 1500)], ids=str)
def test_fp32_factors_of_every_size(ssd, shape):  # noqa: F811
    """Tokens' own factors from 1e-25 to 1e15, one of them 0: a token's dx depends on its own
    alone.  Beside grad_bound: what planes scaled to 2^14 resolve, half of 2^-24 there, so
    2^-39 of the largest W and of 1 for dz; 2^-38 of the largest g x (taken to 2^13 at
    least).  The sum of a token's |dz| is at most 2, that of a word's at most one a token."""
    x, w, t, n = loss_case(shape, "fp32", "some")
    rows, d, V = shape
    g = n(rows) * 10.0 ** (torch.rand(rows, device="cuda") * 40 - 25)
    g[5] = 0.0
    lse = ssd.linear_cross_entropy_forward(x, w, t)[1]
    live = R.cross_entropy(x, w, t)[2]
    z, top = R.logit_bound(x, w, F32, live), float(lse.abs().max())
    dx, dw, ax, aw = R.cross_entropy_backward(x, w, t, g)
    gl = torch.where(live, g, 0.0).double().abs()[:, None]
    gx = gl * x.double().abs()
    off_x = gl * 2.0 ** -39 * (w.double().abs().sum(0) + 2 * w.double().abs().max())
    off_w = 2.0 ** -39 * gx.sum(0) + 2.0 ** -38 * gx.max() * rows
    for want in (None, ("dx",), ("dweight",)):
        r = ssd.linear_cross_entropy_backward(x, w, t, lse, g, want=want)
        if want != ("dweight",):
            bound = R.grad_bound(z, top, ax, V, dx, F32) - 1e-30 + off_x
            within(r["dx"], dx, bound, "dx")
            assert (r["dx"][~live | (g == 0)] == 0).all()
        if want != ("dx",):
            within(r["dweight"], dw, R.grad_bound(z, top, aw, rows, dw, F32) + off_w, "dweight")


def test_fp32_factors_at_the_ends_of_the_range(ssd):  # noqa: F811
    """Factors and rows whose product fits where neither's scale would: the bits of the
    same powers of two taken apart."""
    x, w, t, n = loss_case((70, 64, 300), "fp32", "none")
    lse = ssd.linear_cross_entropy_forward(x, w, t)[1]
    g = n(70)
    ref = ssd.linear_cross_entropy_backward(x, w, t, lse, g)
    for k in (-120, 100):
        r = ssd.linear_cross_entropy_backward(x, w, t, lse, g * 2.0 ** k)
        for name in ref:
            within(r[name], ref[name].double() * 2.0 ** k, 2.0 ** -149, name)  # (denormals)
    dx = ssd.linear_cross_entropy_backward(x, w, t, lse, g * 2.0 ** 124, want=("dx",))["dx"]
    assert float(ref["dx"].abs().max()) < 16 and float(g.abs().max()) < 16
    within(dx, ref["dx"].double() * 2.0 ** 124, 0.0, "dx near the range's end")
    g[3], t[4] = float("inf"), 300  # a token's infinity, and a target that is no word
    dx = ssd.linear_cross_entropy_backward(x, w, t, lse, g, want=("dx",))["dx"]
    keep = torch.arange(70, device="cuda") > 4
    assert torch.equal(dx[keep], ref["dx"][keep]) and torch.equal(dx[:3], ref["dx"][:3])
    assert not torch.isfinite(dx[3]).any() and torch.isnan(dx[4]).all()


def test_losses_of_sure_rows(ssd):  # noqa: F811
    """Logits near 1e4 with the target the largest, the next one tens below: a loss of 0 up to
    the rounding of numbers near 1e4 (loss_bound's 2^-22 of lse, 2.4e-3, and the logits'
    own), each row by its own size.  Losing the target, or counting it twice, shows."""
    x = torch.zeros(5, 16, dtype=B16, device="cuda")
    w = torch.zeros(300, 16, dtype=B16, device="cuda")
    w[:, 0] = torch.linspace(-1, 1, 300, device="cuda")
    w[299, 0] = 1
    x[0, 0], x[1, 0] = 1e4, -1e4
    t = torch.full((5,), 299, device="cuda")
    t[1], t[2] = 0, 7
    ref, ref_lse, live = R.cross_entropy(x, w, t)
    loss, lse = ssd.linear_cross_entropy_forward(x, w, t)
    for i in range(5):
        z = R.logit_bound(x[i:i + 1], w, B16, live[i:i + 1])
        off = R.loss_bound(z, 300, ref_lse[i])
        assert float(off) < 0.05
        within(loss[i], ref[i], off, "loss")
        within(lse[i], ref_lse[i], off, "lse")


def test_words_without_a_share(ssd):  # noqa: F811
    """A channel that is 1 in every token makes W's column a bias: -inf there leaves the
    word out, in bf16.  In fp32, in planes, it is a NaN for every token."""
    n = gen(8)
    x, W = n(70, 40, dtype=B16), n(500, 40, scale=0.3, dtype=B16)
    x[:, 0] = 1
    W[::3, 0] = float("-inf")
    t = torch.arange(70, device="cuda") * 6 + 1
    loss, lse = ssd.linear_cross_entropy_forward(x, W, t)
    z = x.double() @ W.double().t()
    ref = torch.logsumexp(z, 1)
    keep = W[:, 0].isfinite()
    off = R.loss_bound(R.logit_bound(x, W[keep], B16, t >= 0), 500, ref)
    within(lse, ref, off, "lse")
    within(loss, ref - z.gather(1, t[:, None])[:, 0], off, "loss")
    assert torch.isnan(ssd.linear_cross_entropy_forward(x.float(), W.float(), t)[0]).all()


# ----------------------------------------------------- orthogonalised updates

@pytest.mark.parametrize("to", ["bf16", "fp32"])
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("size,eps", [(1e-13, 1e-20), (1e-25, 1e-32), (1e-38, 1e-45), (1e12, 1e-7),
                                      (1e20, 1e-7), (1e37, 1e-7)])
def test_updates_of_every_size(ssd, size, eps, io, to):  # noqa: F811
    """Entries whose squares leave fp32 at either end, down to denormals, and a norm beyond
    its range; in stacks beside matrices of usual size, whose bits do not change."""
    for shape in ((70, 130), (3, 200, 90)):
        G = gen(shape[-1])(*shape, scale=size, dtype=IO[io])
        X = ssd.orthogonalize(G, dtype=IO[to], eps=eps)
        assert relative(X, R.orthogonalize(G, eps=eps)) <= R.orth_bound(IO[to], G)
    H = gen(2)(3, 200, 90, dtype=IO[io])
    ref = ssd.orthogonalize(H, dtype=IO[to], eps=eps)
    H[1] = G[1]
    Y = ssd.orthogonalize(H, dtype=IO[to], eps=eps)
    assert torch.equal(Y[::2], ref[::2]) and torch.equal(Y[1], X[1])


@pytest.mark.parametrize("to", ["bf16", "fp32"])
def test_an_update_of_mixed_sizes(ssd, to):  # noqa: F811
    """Rows of 1e-30, 1 and 1e30 in one matrix: its large rows orthogonalised, the others
    what is left of them next to those (their share of the norm is 1e-30)."""
    G = gen(3)(300, 600)
    G[::3] *= 1e-30
    G[1::3] *= 1e30
    X = ssd.orthogonalize(G, dtype=IO[to])
    assert relative(X, R.orthogonalize(G)) <= R.orth_bound(IO[to], G)


@pytest.mark.parametrize("to", ["bf16", "fp32"])
@pytest.mark.parametrize("eps", [1e-7, 1e-30, 1e-37, 1e-45])
def test_updates_of_zeros_and_of_no_numbers(ssd, eps, to):  # noqa: F811
    """Zeros stay zeros whatever eps is; an infinity or a NaN gives NaN, in its matrix."""
    G = torch.zeros(5, 40, 70, device="cuda")
    G[1, 3, 5] = 1e-30
    G[2, 3, 5], G[3, 7, 7], G[4] = float("inf"), float("nan"), 1e38
    G[4, 0, 0] = float("-inf")
    X = ssd.orthogonalize(G, dtype=IO[to], eps=eps)
    assert (X[0] == 0).all() and torch.isfinite(X[1]).all() and torch.isnan(X[2:]).all()


@pytest.mark.parametrize("to", ["bf16", "fp32"])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_no_number_among_large_values(ssd, what, to):  # noqa: F811
    """The one block of a large matrix that holds it has the smallest values otherwise."""
    G = gen(4)(300, 600)
    G[:250] *= 1e37
    G[299, 599] = float(what)
    assert torch.isnan(ssd.orthogonalize(G, dtype=IO[to])).all()


def test_a_stack_between_the_rows_of_another_axis(ssd):  # noqa: F811
    """Matrices whose rows alternate in memory, read and written so."""
    G = gen(1)(3, 40, 72, dtype=B16)
    X = ssd.orthogonalize(G)
    out = torch.zeros(40, 3, 72, dtype=B16, device="cuda").permute(1, 0, 2)
    ssd.orthogonalize(G, out=out)
    assert torch.equal(out, X)
    H = torch.empty(40, 3, 72, dtype=B16, device="cuda").permute(1, 0, 2).copy_(G)
    assert torch.equal(ssd.orthogonalize(H), X)


def test_smoke_decomposes_nothing_on_the_gpu(ssd, monkeypatch):  # noqa: F811
    """The GPU's decompositions come from a library that need not be there."""
    import __graft_entry__ as entry
    for name in ("svd", "svdvals", "qr", "eigh"):
        def on_host(a, *args, real=getattr(torch.linalg, name), **kw):
            assert not a.is_cuda
            return real(a, *args, **kw)
        monkeypatch.setattr(torch.linalg, name, on_host)
    entry._smoke_model(ssd)
