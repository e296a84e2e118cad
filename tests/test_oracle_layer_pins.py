"""Pins of the float64 oracle of the operators around the scan (CPU): closed
forms and hand-worked values of the forwards, central differences for the
gradients, and agreement of the ways a sequence can be cut."""
import numpy as np
import pytest

from oracle import layer as O

RNG = np.random.default_rng


def differences(f, args, name, cot, h=1e-5):
    """d sum(cot . f) / d args[name] by central differences."""
    base = {k: (None if v is None else np.array(v, np.float64)) for k, v in args.items()}
    out = np.zeros_like(base[name])
    for i in np.ndindex(out.shape):
        vals = []
        for sgn in (1, -1):
            a = dict(base)
            a[name] = base[name].copy()
            a[name][i] += sgn * h
            outs = f(a)
            vals.append(sum((c * o).sum() for c, o in zip(cot, outs)))
        out[i] = (vals[0] - vals[1]) / (2 * h)
    return out


# differences of order h^2 with h = 1e-5 and rounding 1e-16 / h: about 1e-9 of
# O(1) values; 1e-6 leaves room for the sums
TOL = dict(rtol=1e-6, atol=1e-7)


def conv_case(W, lengths, seed):
    r = RNG(seed)
    b, L, D = 3, 5, 2
    return dict(x=r.normal(size=(b, L, D)), weight=r.normal(size=(D, W)), bias=r.normal(size=D),
                state=r.normal(size=(b, W - 1, D))), lengths, (b, L, D)


def test_conv_by_hand():
    x = np.array([[[1.0], [2.0], [3.0]]])
    w = np.array([[10.0, 1.0]])
    y, fin = O.causal_conv(x, w, np.array([0.5]), np.array([[[7.0]]]), act=False)
    np.testing.assert_allclose(y[0, :, 0], [71.5, 12.5, 23.5])
    np.testing.assert_allclose(fin, [[[3.0]]])
    np.testing.assert_allclose(O.silu(np.array([0.0, 1.0])), [0.0, 1 / (1 + np.exp(-1.0))])


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_continues_from_its_state(W):
    a, _, (b, L, D) = conv_case(W, None, W)
    y, fin = O.causal_conv(**a)
    for cut in range(1, L):
        y1, mid = O.causal_conv(a["x"][:, :cut], a["weight"], a["bias"], a["state"])
        y2, end = O.causal_conv(a["x"][:, cut:], a["weight"], a["bias"], mid)
        np.testing.assert_allclose(np.concatenate([y1, y2], 1), y)
        np.testing.assert_allclose(end, fin)
    # a length is the same as a shorter sequence
    y3, fin3 = O.causal_conv(**a, lengths=[0, 2, L])
    np.testing.assert_allclose(fin3[0], a["state"][0])
    np.testing.assert_allclose(y3[1, :2], y[1, :2])
    assert not y3[0].any() and not y3[1, 2:].any()


@pytest.mark.parametrize("W,lengths,act", [(2, None, True), (4, [5, 0, 1], True),
                                           (3, [2, 3, 5], False)])
def test_conv_gradients(W, lengths, act):
    a, lengths, (b, L, D) = conv_case(W, lengths, 10 + W)
    r = RNG(99)
    cot = (r.normal(size=(b, L, D)), r.normal(size=(b, W - 1, D)))
    g = O.causal_conv_backward(**a, gy=cot[0], gfinal=cot[1], lengths=lengths, act=act)
    for name in a:
        ref = differences(lambda k: O.causal_conv(**k, lengths=lengths, act=act), a, name, cot)
        np.testing.assert_allclose(g["d" + name], ref, **TOL)


def scan_case(seed, z=True, G=2):
    r = RNG(seed)
    b, L, D, N = 2, 4, 4, 3
    return dict(u=r.normal(size=(b, L, D)), dt=r.normal(size=(b, L, D)),
                A=-np.exp(r.normal(size=(D, N))), B=r.normal(size=(b, L, G, N)),
                C=r.normal(size=(b, L, G, N)), D=r.normal(size=D),
                z=r.normal(size=(b, L, D)) if z else None, dt_bias=r.normal(size=D),
                h0=r.normal(size=(b, D, N)))


def test_scan_by_hand():
    """One channel, one state: h = 0.5 h + u, y = 3 h + 2 u."""
    ln2 = np.log(2.0)
    y, fin = O.selective_scan(np.array([[[1.0], [2.0]]]), np.ones((1, 2, 1)), np.array([[-ln2]]),
                              np.ones((1, 2, 1, 1)), 3 * np.ones((1, 2, 1, 1)), np.array([2.0]),
                              h0=np.array([[[4.0]]]))
    np.testing.assert_allclose(y[0, :, 0], [3 * 3.0 + 2, 3 * 3.5 + 4])
    np.testing.assert_allclose(fin, [[[3.5]]])


def test_scan_with_equal_decays_is_the_per_head_scan():
    """With A equal over the states and channels of a head, the scan is the
    recurrence of the per-head oracle."""
    import oracle
    r = RNG(3)
    b, L, nh, P, S = 2, 5, 2, 3, 4
    x, B, C = r.normal(size=(b, L, nh, P)), r.normal(size=(b, L, 1, S)), r.normal(size=(b, L, 1, S))
    dt, A = np.exp(r.normal(size=(b, L, nh))), -np.exp(r.normal(size=nh))
    D, h0 = r.normal(size=nh), r.normal(size=(b, nh, P, S))
    ref = oracle.recurrence_np(x, dt, A, B, C, D, h0)
    y, fin = O.selective_scan(x.reshape(b, L, nh * P), np.repeat(dt, P, 2),
                              np.repeat(A, P)[:, None].repeat(S, 1), B, C, np.repeat(D, P),
                              h0=h0.reshape(b, nh * P, S))
    ry, rf = (ref["y"], ref["final_state"]) if isinstance(ref, dict) else ref
    np.testing.assert_allclose(y.reshape(b, L, nh, P), ry, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(fin.reshape(b, nh, P, S), rf, rtol=1e-10, atol=1e-12)


def test_scan_continues_from_its_state():
    a = scan_case(5)
    y, fin = O.selective_scan(**a, dt_softplus=True)
    head = {k: (v[:, :1] if k in ("u", "dt", "B", "C", "z") else v) for k, v in a.items()}
    tail = {k: (v[:, 1:] if k in ("u", "dt", "B", "C", "z") else v) for k, v in a.items()}
    y1, mid = O.selective_scan(**head, dt_softplus=True)
    y2, end = O.selective_scan(**{**tail, "h0": mid}, dt_softplus=True)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y)
    np.testing.assert_allclose(end, fin)


@pytest.mark.parametrize("softplus,z,lengths,G", [(True, True, None, 1), (False, False, [4, 1], 2),
                                                  (True, True, [0, 3], 2)])
def test_scan_gradients(softplus, z, lengths, G):
    a = scan_case(11, z, G)
    r = RNG(12)
    cot = (r.normal(size=a["u"].shape), r.normal(size=a["h0"].shape))
    how = dict(lengths=lengths, dt_softplus=softplus)
    g = O.selective_scan_backward(**a, gy=cot[0], gfinal=cot[1], **how)
    for name in a:
        if a[name] is None:
            continue
        ref = differences(lambda k: O.selective_scan(**k, **how), a, name, cot)
        np.testing.assert_allclose(g["d" + name], ref, **TOL)


@pytest.mark.parametrize("gate", ["none", "input", "output"])
@pytest.mark.parametrize("center", [False, True])
def test_norm_and_its_gradients(gate, center):
    r = RNG(21)
    rows, D, groups = 3, 6, 2
    a = dict(x=r.normal(size=(rows, D)), weight=r.normal(size=D), bias=r.normal(size=D),
             z=None if gate == "none" else r.normal(size=(rows, D)))
    how = dict(groups=groups, gate=gate, center=center)
    plain = O.gated_norm(a["x"], np.ones(D), None, None if gate == "none" else a["z"], **how)
    if gate != "output":  # unit mean square, and zero mean when centred
        n = plain.reshape(rows, groups, -1)
        np.testing.assert_allclose((n * n).mean(2), 1.0, atol=1e-3)
        if center:
            np.testing.assert_allclose(n.mean(2), 0.0, atol=1e-12)
    cot = (r.normal(size=(rows, D)),)
    g = O.gated_norm_backward(**a, gy=cot[0], **how)
    for name in a:
        if a[name] is not None:
            ref = differences(lambda k: (O.gated_norm(**k, **how),), a, name, cot)
            np.testing.assert_allclose(g["d" + name], ref, **TOL)


def test_clip_by_hand():
    norm, out = O.clip_grad_norm([np.array([3.0]), np.array([[4.0]]), np.zeros(0)], 2.5, eps=0.0)
    assert norm == 5.0
    np.testing.assert_allclose(out[0], [1.5])
    np.testing.assert_allclose(out[1], [[2.0]])
    assert out[2].size == 0
    _, same = O.clip_grad_norm([np.array([3.0])], 100.0)
    np.testing.assert_allclose(same[0], [3.0])
