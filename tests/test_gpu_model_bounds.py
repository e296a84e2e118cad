"""The operators around a language model's blocks in the debug-bounds build, which checks
every plain global access: no check may fire, and the results stay those of the release
library; and nothing is written beside an output's rows."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def libs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mamba_ssd_forward_gb300 as m
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    path = build.build_debug()
    release = _abi.load()
    debug = _abi.load(path)

    def use(checked):
        _abi._lib = debug if checked else release
        return m

    yield use
    _abi._lib = release


def normal(*shape, seed=0, scale=1.0, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def calls(ssd, io):
    out = []
    for rows, D in ((1, 1), (70, 40), (33, 771), (9, 2560), (300, 512), (4, 9001)):
        x, r = normal(rows, D, dtype=io), normal(rows, D, seed=1)
        w = 1 + normal(D, scale=0.2)
        y, t = ssd.add_norm_forward(x, r, w)
        out += [y, t, *ssd.add_norm_backward(t, w, y, r).values()]
        for block in (0, 32, 128):
            q, s, _ = ssd.add_norm_quantized(x, r, w, block=block)
            out += [q.float(), s]
    for rows, D, V in ((1, 1, 1), (70, 33, 300), (300, 72, 1000)):
        x, W = normal(rows, D, dtype=io), normal(V, D, scale=1 / math.sqrt(D), dtype=io)
        t = torch.arange(rows, device="cuda") * 7 % V
        t[::4] = -100
        loss, lse = ssd.linear_cross_entropy_forward(x, W, t)
        total, _ = ssd.linear_cross_entropy_forward(x, W, t, reduction="mean")
        out += [loss, lse, total, *ssd.linear_cross_entropy_backward(x, W, t, lse).values()]
    for shape in ((1, 1), (40, 77), (300, 129), (2, 260, 600), (2500, 40)):
        for to in (B16, F32):
            out.append(ssd.orthogonalize(normal(*shape, dtype=io), dtype=to))
    return out


@pytest.mark.parametrize("io", [B16, F32], ids=str)
def test_no_check_fires(libs, io):
    ref = calls(libs(False), io)
    ssd = libs(True)
    got = calls(ssd, io)
    ssd.device_error()  # raises if a check fired
    libs(False)
    for p, q in zip(got, ref):
        assert torch.equal(p, q)


@pytest.mark.parametrize("D", [40, 41, 2560, 2563])
def test_nothing_is_written_beside_the_rows(libs, D):
    ssd = libs(False)

    def frame(dtype, *shape):
        """Rows in the middle of wider ones, with rows before and behind."""
        base = torch.full((shape[0] + 2, shape[1] + 24), 7.0, device="cuda").to(dtype)
        return base, base[1:-1, 8:8 + shape[1]]

    def untouched(base, shape):
        base = base.float().clone()
        base[1:-1, 8:8 + shape[1]] = 7.0
        return bool((base == 7.0).all())

    x, r, w = normal(50, D, dtype=B16), normal(50, D), 1 + normal(D, scale=0.2)
    for quantised in (False, True):
        by, y = frame(torch.float8_e4m3fn if quantised else B16, 50, D)
        bt, t = frame(F32, 50, D)
        if quantised:
            ssd.add_norm_quantized(x, r, w, q=y, total=t)
        else:
            ssd.add_norm_forward(x, r, w, y=y, total=t)
        assert untouched(by, (50, D)) and untouched(bt, (50, D))
    for to in (B16, F32):
        bo, o = frame(to, 50, D)
        ssd.orthogonalize(normal(50, D, dtype=B16), out=o)
        assert untouched(bo, (50, D))
