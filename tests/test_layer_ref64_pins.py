"""The float64 torch references of the convolution and the scan agree with the
numpy oracle (CPU)."""
import numpy as np
import pytest
import torch

import layer_ref64 as R
from layer_cases import conv_inputs, scan_inputs
from oracle import layer as O

TOL = dict(rtol=1e-9, atol=1e-11)  # the same formulas in 64 bits, sums in another order


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    """The seeded inputs are made for the device; here they stay on the host."""
    to, arange = torch.Tensor.to, torch.arange
    monkeypatch.setattr(torch.Tensor, "to", lambda t, a, *r, **k:
                        t if a == "cuda" else to(t, a, *r, **k))
    monkeypatch.setattr(torch, "arange", lambda *a, device=None, **k: arange(*a, **k))


def host(kw):
    return {k: None if v is None else v.double().numpy() for k, v in kw.items()}


def same(got, ref):
    for k, r in ref.items():
        if r is not None:
            np.testing.assert_allclose(got[k].numpy(), r, **TOL, err_msg=k)


@pytest.mark.parametrize("lengths", [None, [7, 0, 2]])
@pytest.mark.parametrize("W,act,state,bias", [(4, True, True, True), (2, False, True, False),
                                              (3, True, False, True)])
def test_conv(lengths, W, act, state, bias):
    a, gy, gf = conv_inputs(3, 7, 5, W, "fp32", seed=W, state=state, bias=bias)
    y, fin = R.causal_conv(**a, lengths=lengths, act=act)
    yr, fr = O.causal_conv(**host(a), lengths=lengths, act=act)
    same({"y": y, "fin": fin}, {"y": yr, "fin": fr})
    for g in (gf, None):
        same(R.causal_conv_backward(**a, gy=gy, gfinal=g, lengths=lengths, act=act),
             O.causal_conv_backward(**host(a), gy=gy.numpy(), gfinal=None if g is None else
                                    g.numpy(), lengths=lengths, act=act))


@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
@pytest.mark.parametrize("G,softplus,more", [(1, True, {}), (2, False, {"z": False}),
                                             (3, True, {"h0": False, "skip": False}),
                                             (1, True, {"bias": False})])
def test_scan(lengths, G, softplus, more):
    a, gy, gf = scan_inputs(3, 9, 6, 5, G, "fp32", seed=G, **more)
    how = dict(lengths=lengths, dt_softplus=softplus)
    y, fin = R.selective_scan(**a, **how)
    yr, fr = O.selective_scan(**host(a), **how)
    same({"y": y, "fin": fin}, {"y": yr, "fin": fr})
    for g in (gf, None):
        same(R.selective_scan_backward(**a, gy=gy, gfinal=g, **how),
             O.selective_scan_backward(**host(a), gy=gy.numpy(), gfinal=None if g is None else
                                       g.numpy(), **how))
