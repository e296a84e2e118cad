"""The operators around a language model's blocks where their types, panes and number
ranges end, on the GPU against their float64 definitions.  Bounds: tests/model_ref64.py."""
import pytest
import torch

import model_ref64 as R
from test_gpu_model import F32, check_loss, loss_case, ssd, within  # noqa: F401

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
    g[3], t[4] = float("inf"), 300  # a token's infinity, and a target that is no word
    dx = ssd.linear_cross_entropy_backward(x, w, t, lse, g, want=("dx",))["dx"]
    keep = torch.arange(70, device="cuda") > 4
    assert torch.equal(dx[keep], ref["dx"][keep]) and torch.equal(dx[:3], ref["dx"][:3])
    assert not torch.isfinite(dx[3]).any() and torch.isnan(dx[4]).all()
