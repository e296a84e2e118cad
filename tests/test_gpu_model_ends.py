"""The operators around a language model's blocks where their types, panes and number
ranges end, on the GPU against their float64 definitions.  Bounds: tests/model_ref64.py."""
import pytest

from test_gpu_model import check_loss, loss_case, ssd  # noqa: F401

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
