"""Host-side refusals of the operators around the scan: bad dims, types,
pointers, strides and workspaces are rejected before anything is launched (no
GPU needed), and the Python calls name what is wrong."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    return _abi.load()


@pytest.fixture(scope="module")
def abi():
    from mamba_ssd_forward_gb300 import _abi
    return _abi


OK = 1 << 20          # aligned, never dereferenced: the checks fail first
ODD = (1 << 20) + 1


def seq(abi, data=OK, bs=4096, ts=64):
    return abi.SsdSeq(data, bs, ts)


def conv(abi, **kw):
    return abi.SsdConvDims(**{**dict(batch=2, seqlen=8, channels=64, width=4, activation=1), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(channels=0), 1), (dict(width=0), 1),
    (dict(activation=2), 1), (dict(width=1), 2), (dict(width=5), 2), (dict(batch=65536), 2),
    (dict(seqlen=1 << 31), 2)])
def test_conv_dims(lib, abi, kw, code):
    d, x = conv(abi, **kw), seq(abi)
    assert lib.ssd_causal_conv(d, 1, x, OK, None, None, None, x, None, None) == code
    assert lib.ssd_causal_conv_backward_workspace_size(d, 1) == 0
    assert lib.ssd_causal_conv_backward(d, 1, x, OK, None, None, x, None, None, x, OK, None,
                                        None, OK, 1 << 40, None) == code
    if "seqlen" not in kw:
        one = conv(abi, **{**kw, "seqlen": 1})
        assert lib.ssd_causal_conv_step(one, 1, x, OK, None, OK, x, None) == code


def test_conv_pointers(lib, abi):
    d, x = conv(abi), seq(abi)
    good = [x, OK, None, None, None, x, None]  # x weight bias state lengths y final_state
    for i, v in enumerate(good):
        for bad in ([None] if v is not None else []) + [seq(abi, ODD) if i in (0, 5) else ODD]:
            a = list(good)
            a[i] = bad
            assert lib.ssd_causal_conv(d, 1, *a, None) == 1, (i, bad)
    assert lib.ssd_causal_conv(d, 1, seq(abi, bs=-1), *good[1:], None) == 1
    assert lib.ssd_causal_conv(d, 1, seq(abi, ts=-1), *good[1:], None) == 1
    assert lib.ssd_causal_conv(d, 1, seq(abi, ts=1 << 60), *good[1:], None) == 1
    assert lib.ssd_causal_conv(d, 7, *good, None) == 1
    assert lib.ssd_causal_conv(None, 1, *good, None) == 1
    need = lib.ssd_causal_conv_backward_workspace_size(d, 1)
    assert need > 0
    back = [x, OK, None, None, x, None, None, x, OK, None, None]
    for ws, n in ((None, need), (OK, need - 1), (OK + 16, need)):
        assert lib.ssd_causal_conv_backward(d, 1, *back, ws, n, None) == 1
    # a token call takes one token and needs its state
    assert lib.ssd_causal_conv_step(d, 1, x, OK, None, OK, x, None) == 1
    assert lib.ssd_causal_conv_step(conv(abi, seqlen=1), 1, x, OK, None, None, x, None) == 1


def scan(abi, **kw):
    return abi.SsdScanDims(**{**dict(batch=2, seqlen=8, channels=64, dstate=16, ngroups=2,
                                     dt_softplus=1), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(channels=0), 1), (dict(dstate=0), 1),
    (dict(ngroups=0), 1), (dict(ngroups=3), 1), (dict(dt_softplus=2), 1), (dict(dstate=65), 2),
    (dict(batch=65536), 2), (dict(ngroups=1 << 17, channels=1 << 18), 2)])
def test_scan_dims(lib, abi, kw, code):
    d, x = scan(abi, **kw), seq(abi)
    ins = [x, x, OK, x, x, None, None, None]
    assert lib.ssd_selective_scan(d, 1, *ins, None, None, x, None, OK, 1 << 40, None) == code
    assert lib.ssd_selective_scan_backward_workspace_size(d, 1) == 0
    g = abi.SsdScanGrads(du=x, ddt=x, dB=x, dC=x)
    assert lib.ssd_selective_scan_backward(d, 1, *ins, None, x, None, None, g, OK, 1 << 40,
                                           None) == code
    if "seqlen" not in kw:
        assert lib.ssd_selective_scan_step(scan(abi, **{**kw, "seqlen": 1}), 1, *ins, OK, x,
                                           None) == code


def test_scan_pointers(lib, abi):
    d, x = scan(abi), seq(abi)
    good = [x, x, OK, x, x, None, None, None, None, None, x, None]
    views = (0, 1, 3, 4, 6, 10)  # u dt B C z y
    need = lib.ssd_selective_scan_workspace_size(d, 1)
    for i, v in enumerate(good):
        for bad in ([None] if v is not None else []) + [seq(abi, ODD) if i in views else ODD]:
            a = list(good)
            a[i] = bad
            assert lib.ssd_selective_scan(d, 1, *a, OK, max(need, 256), None) == 1, (i, bad)
    assert lib.ssd_selective_scan_step(d, 1, *good[:8], OK, x, None) == 1  # seqlen 8
    assert lib.ssd_selective_scan_step(scan(abi, seqlen=1), 1, *good[:8], None, x, None) == 1
    need = lib.ssd_selective_scan_backward_workspace_size(d, 1)
    assert need > 0
    full = dict(du=x, ddt=x, dB=x, dC=x)

    def back(g, ws=OK, n=need):
        return lib.ssd_selective_scan_backward(d, 1, *good[:9], x, None, None, g, ws, n, None)

    for k in full:  # required
        assert back(abi.SsdScanGrads(**{j: v for j, v in full.items() if j != k})) == 1
    assert back(None) == 1
    assert back(abi.SsdScanGrads(**full, dz=x)) == 1  # a gradient of an absent gate
    assert back(abi.SsdScanGrads(**full, dA=ODD)) == 1
    full = abi.SsdScanGrads(**full)
    assert back(full, None) == 1 and back(full, OK, need - 1) == 1 and back(full, OK + 16) == 1


def norm(abi, **kw):
    return abi.SsdNormDims(**{**dict(batch=2, seqlen=8, channels=64, ngroups=2, eps=1e-5, gate=1,
                                     center=0), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(channels=0), 1), (dict(ngroups=0), 1),
    (dict(ngroups=3), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(gate=3), 1), (dict(gate=-1), 1), (dict(center=2), 1),
    (dict(channels=1 << 18, ngroups=2), 2)])
def test_norm_dims(lib, abi, kw, code):
    d, x = norm(abi, **kw), seq(abi)
    assert lib.ssd_gated_norm(d, 1, x, OK, None, x, x, None) == code
    assert lib.ssd_gated_norm_backward_workspace_size(d, 1) == 0
    assert lib.ssd_gated_norm_backward(d, 1, x, OK, None, x, x, x, x, OK, None, OK, 1 << 40,
                                       None) == code


def test_norm_pointers(lib, abi):
    d, x = norm(abi), seq(abi)
    good = [x, OK, None, x, x]
    for i in range(5):
        for bad in ([None] if good[i] is not None else []) + [ODD if i in (1, 2) else
                                                             seq(abi, ODD)]:
            a = list(good)
            a[i] = bad
            assert lib.ssd_gated_norm(d, 1, *a, None) == 1, (i, bad)
    # a gate without a mode that reads it
    assert lib.ssd_gated_norm(norm(abi, gate=0), 1, *good, None) == 1
    need = lib.ssd_gated_norm_backward_workspace_size(d, 1)
    args = [x, OK, None, x, x, x, x, OK, None]
    assert lib.ssd_gated_norm_backward(d, 1, *args, OK, need - 1, None) == 1
    args[6] = None  # dz is required with a gate
    assert lib.ssd_gated_norm_backward(d, 1, *args, OK, need, None) == 1


def test_clip_arguments(lib, abi):
    def table(**kw):
        t = (abi.SsdGrad * 1)()
        t[0] = tuple({**dict(src=OK, dst=OK, n=10, dtype=0), **kw}.values())
        return t

    def call(t, n=1, max_norm=1.0, eps=1e-6, out=OK, ws=OK, size=1 << 20):
        return lib.ssd_clip_grad_norm(t, n, max_norm, eps, out, ws, size, None)

    assert lib.ssd_clip_grad_norm_workspace_size(table(), 1) > 0
    for bad in (dict(n=-1), dict(dtype=2), dict(src=None), dict(dst=None), dict(src=ODD),
                dict(dst=ODD)):
        assert call(table(**bad)) == 1, bad
        assert lib.ssd_clip_grad_norm_workspace_size(table(**bad), 1) == 0
    nan = float("nan")
    for kw in (dict(n=-1), dict(max_norm=-1.0), dict(max_norm=nan), dict(eps=-1.0),
               dict(eps=nan), dict(eps=float("inf")), dict(out=None), dict(out=ODD),
               dict(ws=None), dict(size=1)):
        assert call(table(), **kw) == 1, kw
    assert call(None) == 1


def test_python_calls_say_what_is_wrong():
    import mamba_ssd_forward_gb300 as ssd
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.causal_conv_forward(x, w)
    with pytest.raises(TypeError, match="x must be"):
        ssd.causal_conv_forward(x.half(), w)
    with pytest.raises(ValueError, match="activation"):
        ssd.causal_conv_forward(x, w, activation="relu")
    with pytest.raises(ValueError, match=r"\[b, L, D\]"):
        ssd.causal_conv_forward(x[0], w)
    with pytest.raises(ValueError, match="gy"):
        ssd.causal_conv_backward(x, w)
    A, B = torch.zeros(8, 4), torch.zeros(2, 5, 1, 4)
    with pytest.raises(ValueError, match="must be"):
        ssd.selective_scan_forward(x, x, A, B[0], B)
    with pytest.raises(ValueError, match="state"):
        ssd.selective_scan_step(x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], None, None, None, None)
    with pytest.raises(ValueError, match="gate"):
        ssd.gated_norm_forward(x, torch.zeros(8), gate="both")
    with pytest.raises(ValueError, match="CUDA"):
        ssd.clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError, match="outputs"):
        ssd.clip_grad_norm([x], 1.0, out=[])
    with pytest.raises(ValueError, match="no gradients"):
        ssd.clip_grad_norm([], 1.0)
