"""Host-side refusals of the operators around a language model's blocks: bad dims, types,
pointers, strides and workspaces are rejected before anything is launched (no GPU
needed), and the Python calls name what is wrong."""
import pytest
import torch

import mamba_ssd_forward_gb300 as ssd

OK = 1 << 20  # aligned, never dereferenced: the checks fail first
ODD = (1 << 20) + 1
BIG = 1 << 50


@pytest.fixture(scope="module")
def abi():
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    return _abi


@pytest.fixture(scope="module")
def lib(abi):
    return abi.load()


def seq(abi, data=OK, bs=4096, ts=64):
    return abi.SsdSeq(data, bs, ts)


def norm(abi, **kw):
    return abi.SsdAddNormDims(**{**dict(batch=2, seqlen=8, channels=64, eps=1e-5), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(channels=0), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(channels=16385), 2), (dict(batch=1 << 20, seqlen=1 << 20), 2)])
def test_add_norm_dims(lib, abi, kw, code):
    d, x = norm(abi, **kw), seq(abi)
    assert lib.ssd_add_norm(d, 1, 0, x, x, OK, x, x, None) == code
    assert lib.ssd_add_norm_quantized(d, 1, 0, 128, x, x, OK, x, OK, x, None) == code
    assert lib.ssd_add_norm_backward_workspace_size(d, 1, 0) == 0
    assert lib.ssd_add_norm_backward(d, 1, 0, x, OK, x, x, x, x, OK, OK, BIG, None) == code


def test_add_norm_arguments(lib, abi):
    d, x = norm(abi), seq(abi)
    odd, shared = seq(abi, ODD), seq(abi, ts=63)
    good = [x, x, OK, x, x]  # x residual weight y total
    for i, bad in ((0, None), (0, odd), (1, odd), (2, None), (2, ODD), (3, None), (3, odd),
                   (3, shared), (4, odd), (4, shared), (0, seq(abi, bs=-1)),
                   (1, seq(abi, ts=1 << 60))):
        a = list(good)
        a[i] = bad
        assert lib.ssd_add_norm(d, 1, 0, *a, None) == 1, (i, bad)
    for io, stream in ((7, 0), (1, 7), (0, 1)):  # a bf16 stream under fp32 activations
        assert lib.ssd_add_norm(d, io, stream, *good, None) == 1
    q = [x, x, OK, x, OK, x]  # x residual weight q scales total
    for block in (1, 16, 96, 256, -1):
        assert lib.ssd_add_norm_quantized(d, 1, 0, block, *q, None) == 1
    for i, bad in ((3, None), (3, shared), (4, None), (4, ODD)):
        a = list(q)
        a[i] = bad
        assert lib.ssd_add_norm_quantized(d, 1, 0, 128, *a, None) == 1, (i, bad)
    need = lib.ssd_add_norm_backward_workspace_size(d, 1, 0)
    assert need > 0
    back = [x, OK, x, x, x, x, OK]  # total weight gy gtotal dx dresidual dweight
    for ws, n in ((None, need), (OK, need - 1), (OK + 16, need)):
        assert lib.ssd_add_norm_backward(d, 1, 0, *back, ws, n, None) == 1
    for i, bad in ((0, None), (1, None), (2, None), (3, odd), (4, shared), (5, shared), (6, ODD)):
        a = list(back)
        a[i] = bad
        assert lib.ssd_add_norm_backward(d, 1, 0, *a, OK, need, None) == 1, (i, bad)
    # nothing asked for: nothing to do
    assert lib.ssd_add_norm_backward(d, 1, 0, *back[:4], None, None, None, None, 0, None) == 0


def loss(abi, **kw):
    return abi.SsdLossDims(**{**dict(batch=2, seqlen=8, channels=64, vocab=100, ignore_index=-100,
                                     reduction=0), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(channels=0), 1), (dict(vocab=0), 1),
    (dict(reduction=3), 1), (dict(reduction=-1), 1), (dict(channels=65537), 2),
    (dict(vocab=(1 << 24) + 1), 2), (dict(batch=1 << 15, seqlen=1 << 16), 2),
    (dict(batch=1, seqlen=1 << 29, vocab=1 << 20), 2)])
def test_loss_dims(lib, abi, kw, code):
    d, x = loss(abi, **kw), seq(abi)
    total = OK if d.reduction else None
    assert lib.ssd_linear_cross_entropy_workspace_size(d, 1, x) == 0
    assert lib.ssd_linear_cross_entropy(d, 1, x, x, OK, OK, total, OK, OK, BIG, None) == code
    assert lib.ssd_linear_cross_entropy_backward_workspace_size(d, 1, x) == 0
    assert lib.ssd_linear_cross_entropy_backward(d, 1, x, x, OK, OK, OK, x, OK, OK, BIG,
                                                 None) == code


def test_loss_arguments(lib, abi):
    d, x = loss(abi), seq(abi)
    odd, shared = seq(abi, ODD), seq(abi, ts=63)
    need = lib.ssd_linear_cross_entropy_workspace_size(d, 1, x)
    assert need > 0
    # x weight targets loss total lse
    good = [x, x, OK, OK, None, OK]
    for i, bad in ((0, None), (0, odd), (1, None), (1, odd), (1, seq(abi, ts=-1)), (2, None),
                   (2, OK + 4), (3, None), (3, ODD), (4, OK), (5, None), (5, ODD)):
        a = list(good)
        a[i] = bad
        assert lib.ssd_linear_cross_entropy(d, 1, *a, OK, BIG, None) == 1, (i, bad)
    for ws, n in ((None, need), (OK, need - 1), (OK + 16, need)):
        assert lib.ssd_linear_cross_entropy(d, 1, *good, ws, n, None) == 1
    # a reduction needs its result
    assert lib.ssd_linear_cross_entropy(loss(abi, reduction=2), 1, *good, OK, BIG, None) == 1
    need = lib.ssd_linear_cross_entropy_backward_workspace_size(d, 1, x)
    assert need > 0
    back = [x, x, OK, OK, OK, x, OK]  # x weight targets lse gloss dx dweight
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (4, ODD), (5, shared), (6, ODD)):
        a = list(back)
        a[i] = bad
        assert lib.ssd_linear_cross_entropy_backward(d, 1, *a, OK, BIG, None) == 1, (i, bad)
    for ws, n in ((None, need), (OK, need - 1), (OK + 16, need)):
        assert lib.ssd_linear_cross_entropy_backward(d, 1, *back, ws, n, None) == 1
    assert lib.ssd_linear_cross_entropy_backward(d, 1, *back[:5], None, None, OK, BIG, None) == 0
    # W that TMA can take as it is needs no room for a copy
    assert lib.ssd_linear_cross_entropy_workspace_size(d, 1, seq(abi, OK + 2)) > \
        lib.ssd_linear_cross_entropy_workspace_size(d, 1, x)


def orth(abi, **kw):
    return abi.SsdOrthDims(**{**dict(count=2, rows=64, cols=48, steps=5, a=3.4445, b=-4.775,
                                     c=2.0315, eps=1e-7), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(count=0), 1), (dict(rows=0), 1), (dict(cols=0), 1), (dict(steps=0), 1),
    (dict(steps=101), 1), (dict(a=float("inf")), 1), (dict(b=float("nan")), 1), (dict(eps=0.0), 1),
    (dict(eps=float("nan")), 1), (dict(count=32768), 2), (dict(rows=(1 << 20) + 1), 2),
    (dict(cols=(1 << 20) + 1), 2), (dict(count=30000, rows=1 << 17, cols=1 << 17), 2)])
def test_orth_dims(lib, abi, kw, code):
    d, x = orth(abi, **kw), seq(abi)
    assert lib.ssd_orthogonalize_workspace_size(d, 1, 1) == 0
    assert lib.ssd_orthogonalize(d, 1, 1, x, x, OK, BIG, None) == code


def test_orth_arguments(lib, abi):
    d, x = orth(abi), seq(abi)
    need = lib.ssd_orthogonalize_workspace_size(d, 1, 1)
    assert 0 < need < lib.ssd_orthogonalize_workspace_size(d, 1, 0)  # two planes of A and B
    for u, r in ((None, x), (seq(abi, ODD), x), (x, None), (x, seq(abi, ODD)),
                 (x, seq(abi, ts=47)), (x, seq(abi, bs=64)), (seq(abi, bs=-1), x)):
        assert lib.ssd_orthogonalize(d, 1, 1, u, r, OK, BIG, None) == 1
    for ws, n in ((None, need), (OK, need - 1), (OK + 16, need)):
        assert lib.ssd_orthogonalize(d, 1, 1, x, x, ws, n, None) == 1
    assert lib.ssd_orthogonalize(d, 7, 1, x, x, OK, BIG, None) == 1
    assert lib.ssd_orthogonalize(d, 1, 7, x, x, OK, BIG, None) == 1


# ----------------------------------------------- what the Python calls say

class OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:1; never dereferenced."""

    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


def far(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


B16, I64 = torch.bfloat16, torch.int64


def refusals():
    x, w, r = far(4, 8, dtype=B16), far(8), far(4, 8)
    W, t = far(10, 8, dtype=B16), far(4, dtype=I64)
    G = far(6, 5, dtype=B16)
    f, q, b = ssd.add_norm_forward, ssd.add_norm_quantized, ssd.add_norm_backward
    ce, ceb, o = (ssd.linear_cross_entropy_forward, ssd.linear_cross_entropy_backward,
                  ssd.orthogonalize)
    return {
        "x half": (lambda: f(far(4, 8, dtype=torch.half), r, w), TypeError, "x must be float32"),
        "x 1-d": (lambda: f(far(8), far(8), w), ValueError, "tokens, D"),
        "x empty": (lambda: f(far(0, 8), far(0, 8), w), ValueError, "must not be empty"),
        "residual type": (lambda: f(far(4, 8), far(4, 8, dtype=B16), w), TypeError, "residual"),
        "residual shape": (lambda: f(x, far(4, 9), w), ValueError, "residual must have shape"),
        "weight": (lambda: f(x, r, far(9)), ValueError, "weight must have shape"),
        "weight type": (lambda: f(x, r, far(8, dtype=B16)), TypeError, "weight must be"),
        "transposed": (lambda: f(far(8, 4, dtype=B16).t(), r, w), ValueError, "dense along"),
        "host": (lambda: f(torch.zeros(4, 8, dtype=B16), r, w), ValueError, "CUDA tensor"),
        "y is residual": (lambda: f(far(4, 8), r, w, y=r), ValueError, "must not be the memory"),
        "y is total": (lambda z=far(4, 8): f(far(4, 8), r, w, y=z, total=z), ValueError,
                       "must not be the memory"),
        "y rows": (lambda: f(x, r, w, y=far(1, 8, dtype=B16).expand(4, 8)), ValueError,
                   "must not share"),
        "block": (lambda: q(x, r, w, block=16), ValueError, "block must be"),
        "scales": (lambda: q(x, r, w, scales=far(4, 2)), ValueError, "scales must have shape"),
        "q type": (lambda: q(x, r, w, q=far(4, 8)), TypeError, "q must be"),
        "gradient": (lambda: b(r, w, x, want=("dz",)), ValueError, "no gradient 'dz'"),
        "gtotal": (lambda: b(r, w, x, x), TypeError, "gtotal must be"),
        "residual": (lambda: ssd.add_norm(x, None, w), ValueError, "residual is required"),
        "reduction": (lambda: ce(x, W, t, reduction="max"), ValueError, "reduction must be"),
        "targets type": (lambda: ce(x, W, far(4, dtype=torch.int32)), TypeError,
                         "targets must be"),
        "targets shape": (lambda: ce(x, W, far(5, dtype=I64)), ValueError, "targets must have"),
        "weight width": (lambda: ce(x, far(10, 9, dtype=B16), t), ValueError, "weight must have"),
        "loss weight type": (lambda: ce(x, far(10, 8), t), TypeError, "weight must be"),
        "lse": (lambda: ceb(x, W, t, far(5)), ValueError, "lse must have shape"),
        "gloss": (lambda: ceb(x, W, t, far(4), far(4), reduction="mean"), ValueError, "gloss"),
        "loss gradient": (lambda: ceb(x, W, t, far(4), want=("dbias",)), ValueError, "'dbias'"),
        "update 1-d": (lambda: o(far(5)), ValueError, "update must be"),
        "update empty": (lambda: o(far(0, 5)), ValueError, "not empty"),
        "result type": (lambda: o(G, dtype=torch.half), TypeError, "result must be"),
        "out shape": (lambda: o(G, out=far(5, 6, dtype=B16)), ValueError, "out must have shape"),
        "out type": (lambda: o(G, dtype=B16, out=far(6, 5)), TypeError, "out must be"),
        "workspace": (lambda: o(G, workspace=far(16, dtype=torch.uint8)), ValueError,
                      "16 bytes, "),
        "device": (lambda: f(x, r, w), ValueError, "current device"),
    }


@pytest.mark.parametrize("name", list(refusals()))
def test_refusals_by_name(abi, name, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    real = torch.empty

    def empty(*a, **k):  # outputs on the tensors' device, which is not there
        k.pop("device", None)
        return real(*a, **k).as_subclass(OnDevice)

    monkeypatch.setattr(torch, "empty", empty)
    call, kind, words = refusals()[name]
    with pytest.raises(kind, match=words):
        call()
