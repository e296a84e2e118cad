"""The float64 definitions of the operators around a language model's blocks, pinned by
values worked out by hand, differences of the forward formulas, and closed forms."""
import math

import pytest
import torch

import model_ref64 as R

D64 = torch.float64


def normal(*shape, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=D64)


def difference(f, x, h=1e-6):
    """df/dx of a scalar function, a component at a time."""
    out = torch.empty_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + h
        up = float(f())
        flat[i] = keep - h
        o[i] = (up - float(f())) / (2 * h)
        flat[i] = keep
    return out


def test_norm_by_hand():
    y, t = R.add_norm(torch.tensor([[1.0, 2.0]]), torch.tensor([[2.0, 2.0]]),
                      torch.tensor([1.0, 0.5]), eps=1e-30)
    assert t.tolist() == [[3.0, 4.0]]
    r = 1 / math.sqrt(12.5)  # mean of 9 and 16
    assert torch.allclose(y, torch.tensor([[3 * r, 2 * r]], dtype=D64))


def test_norm_gradients_by_differences():
    t, w, gy, gt = normal(3, 7), 1 + normal(7, seed=1), normal(3, 7, seed=2), normal(3, 7, seed=3)
    dt, dw = R.add_norm_backward(t, w, gy, gt)

    def f():
        y, total = R.add_norm(t, None, w)
        return (y * gy).sum() + (total * gt).sum()

    assert torch.allclose(dt, difference(f, t), atol=1e-7)
    assert torch.allclose(dw, difference(f, w), atol=1e-7)


def test_cross_entropy_by_hand():
    # logits 0 and log 3: probabilities 1/4 and 3/4
    x, w = torch.tensor([[1.0], [1.0], [5.0]]), torch.tensor([[0.0], [math.log(3.0)]])
    loss, lse, live = R.cross_entropy(x, w, torch.tensor([0, 1, -100]))
    assert torch.allclose(loss, torch.tensor([math.log(4), math.log(4 / 3), 0.0], dtype=D64))
    assert live.tolist() == [True, True, False] and float(lse[2]) == 0.0
    assert math.isnan(float(R.cross_entropy(x, w, torch.tensor([2, 0, 0]))[0][0]))
    dx, dw, _, _ = R.cross_entropy_backward(x, w, torch.tensor([0, 1, -100]), torch.ones(3))
    assert torch.allclose(dw[:, 0], torch.tensor([-0.75 + 0.25, 0.75 - 0.25], dtype=D64))
    assert float(dx[2, 0]) == 0.0


def test_cross_entropy_gradients_by_differences():
    x, w, g = normal(5, 4), normal(9, 4, seed=1), normal(5, seed=2)
    t = torch.tensor([3, -100, 0, 8, 3])
    dx, dw, ax, aw = R.cross_entropy_backward(x, w, t, g)

    def f():
        return (R.cross_entropy(x, w, t)[0] * g).sum()

    assert torch.allclose(dx, difference(f, x), atol=1e-7)
    assert torch.allclose(dw, difference(f, w), atol=1e-7)
    assert (ax >= dx.abs()).all() and (aw >= dw.abs()).all()


@pytest.mark.parametrize("shape", [(6, 9), (9, 6), (5, 5), (2, 4, 7)])
def test_orthogonalize_is_its_products(shape):
    a, b, c = 3.4445, -4.7750, 2.0315
    G = normal(*shape)
    out = []
    for g in G.reshape(-1, *shape[-2:]):
        x = g / (g.norm() + 1e-7)
        for _ in range(5):
            s = x @ x.t()
            x = a * x + (b * s + c * s @ s) @ x
        out.append(x)
    assert torch.allclose(R.orthogonalize(G), torch.stack(out).reshape(shape), atol=1e-10)


def test_orthogonalize_of_a_rotation_is_one_number():
    q = torch.linalg.qr(normal(4, 4))[0]
    s = 0.5  # singular values of q / |q|
    for _ in range(2):
        s = 3.4445 * s - 4.775 * s ** 3 + 2.0315 * s ** 5
    assert torch.allclose(R.orthogonalize(q, steps=2, eps=0.0), s * q)
