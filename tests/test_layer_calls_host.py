"""Host side of the calls around the scan (no GPU needed): what they refuse by
name before anything is launched, and what they ask of the library."""
import pytest
import torch

import mamba_ssd_forward_gb300 as ssd


class OnDevice1(torch.Tensor):
    """A host tensor that says it is on cuda:1; never dereferenced."""

    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


def far(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)


def _calls():
    x, w, tok = far(2, 5, 8), far(8, 4), far(2, 8)
    A, B = far(8, 4), far(2, 5, 1, 4)
    big = far(1 << 20, dtype=torch.uint8)
    x4, dt, B4, D1 = far(1, 64, 2, 64), far(1, 64, 2), far(1, 64, 1, 64), far(2)
    return {
        "conv": lambda: ssd.causal_conv_forward(x, w, y=far(2, 5, 8), return_final_state=False),
        "conv_step": lambda: ssd.causal_conv_step(tok, w, None, far(2, 3, 8), y=far(2, 8)),
        "scan": lambda: ssd.selective_scan_forward(x, x, A, B, B, y=far(2, 5, 8), workspace=big,
                                                   return_final_state=False),
        "scan_step": lambda: ssd.selective_scan_step(tok, tok, A, B[:, 0], B[:, 0], None, None,
                                                     None, far(2, 8, 4), y=far(2, 8)),
        "norm": lambda: ssd.gated_norm_forward(x, far(8), gate="none", y=far(2, 5, 8)),
        "forward": lambda: ssd.forward(x4, dt, D1, B4, B4, chunk=64, y=far(1, 64, 2, 64),
                                       workspace=big, return_final_state=False),
        "decode_step": lambda: ssd.decode_step(x4[:, 0], dt[:, 0], D1, B4[:, 0], B4[:, 0], None,
                                               far(1, 2, 64, 64), y=far(1, 2, 64)),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    """The library launches on the current device, cuda:0 here."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="cuda:1.*current.*cuda:0"):
        _calls()[name]()


def _differentiated(monkeypatch):
    """(outputs, inputs) of each differentiable call, its kernels replaced by
    host arithmetic of the same shapes."""
    from mamba_ssd_forward_gb300 import layer
    like = torch.zeros_like

    def pair(x, *a, **k):
        return 2.0 * x, like(x)

    monkeypatch.setattr(layer, "causal_conv_forward", pair)
    monkeypatch.setattr(layer, "causal_conv_backward", lambda x, w, *a, **k: {
        "dx": 2.0 * x, "dweight": like(w), "dbias": None, "dstate": None})
    monkeypatch.setattr(layer, "selective_scan_forward", pair)
    monkeypatch.setattr(layer, "selective_scan_backward", lambda u, dt, A, B, C, *a, **k: {
        "du": 2.0 * u, "ddt": like(dt), "dA": like(A), "dB": like(B), "dC": like(C),
        **dict.fromkeys(("dD", "dz", "ddt_bias", "dh0"))})
    monkeypatch.setattr(layer, "gated_norm_forward", lambda x, *a, **k: 2.0 * x)
    monkeypatch.setattr(layer, "gated_norm_backward", lambda x, w, *a, **k: {
        "dx": 2.0 * x, "dweight": like(w), "dbias": None, "dz": None})
    monkeypatch.setattr(ssd, "forward", pair)
    monkeypatch.setattr(ssd, "backward", lambda x, dt, A, B, C, *a, **k: {
        "dx": 2.0 * x, "ddt": like(dt), "dA": like(A), "dB": like(B), "dC": like(C),
        "dD": None, "dh0": None})

    def leaf(*shape):
        return torch.randn(*shape, requires_grad=True)

    x, w, A, B = leaf(2, 5, 8), leaf(8, 4), leaf(8, 4), leaf(2, 5, 1, 4)
    yield "conv", ssd.causal_conv(x, w)[0], x
    yield "scan", ssd.selective_scan(x, x, A, B, B)[0], x
    yield "norm", ssd.gated_norm(x, leaf(8), gate="none"), x
    x4 = leaf(1, 64, 2, 64)
    yield "ssd", ssd.ssd(x4, leaf(1, 64, 2), leaf(2), leaf(1, 64, 1, 64), leaf(1, 64, 1, 64))[0], x4


@pytest.mark.parametrize("which", ["conv", "scan", "norm", "ssd"])
def test_second_derivatives_are_refused(which, monkeypatch):
    """The gradients come from kernels without gradients of their own: asking
    for them raises, also where other terms have some."""
    y, x = next((y, x) for name, y, x in _differentiated(monkeypatch) if name == which)
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    penalty = (g * g).sum() + (x ** 3).sum()
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(penalty, x)


@pytest.mark.parametrize("which", ["conv", "scan", "norm", "ssd"])
def test_first_derivatives_within_a_graph(which, monkeypatch):
    """create_graph alone changes nothing: other terms are differentiated twice."""
    y, x = next((y, x) for name, y, x in _differentiated(monkeypatch) if name == which)
    plain, = torch.autograd.grad(y.sum(), x, retain_graph=True)
    g, = torch.autograd.grad((x ** 3).sum() + y.sum(), x, create_graph=True)
    assert torch.equal(g.detach(), 3 * x.detach() ** 2 + plain)
    h, = torch.autograd.grad((x ** 3).sum(), x, create_graph=True)
    hh, = torch.autograd.grad(h.sum(), x)
    assert torch.allclose(hh, 6 * x.detach())


@pytest.mark.parametrize("fn,args,names", [
    ("causal_conv", dict(x=(2, 5, 8), weight=(8, 4), bias=(8,), state=(2, 3, 8)),
     ("dx", "dweight", "dbias", "dstate")),
    ("selective_scan", dict(u=(2, 5, 8), dt=(2, 5, 8), A=(8, 4), B=(2, 5, 1, 4), C=(2, 5, 1, 4),
                            D=(8,), z=(2, 5, 8), dt_bias=(8,), h0=(2, 8, 4)),
     ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")),
    ("gated_norm", dict(x=(2, 5, 8), weight=(8,), bias=(8,), z=(2, 5, 8)),
     ("dx", "dweight", "dbias", "dz"))])
def test_only_needed_gradients_are_asked_for(fn, args, names, monkeypatch):
    from mamba_ssd_forward_gb300 import layer
    pair = fn != "gated_norm"
    monkeypatch.setattr(layer, fn + "_forward", lambda x, *a, **k:
                        (2.0 * x, torch.zeros(3)) if pair else 2.0 * x)
    asked = []

    def backward(*a, want=None, **k):
        asked.append(want)
        return {n: torch.ones(s) for n, s in zip(names, args.values())}

    monkeypatch.setattr(layer, fn + "_backward", backward)
    for frozen in ((names[1],), names[1:], (names[0], names[-1])):
        leaf = {k: torch.randn(s, requires_grad=n not in frozen)
                for (k, s), n in zip(args.items(), names)}
        y = getattr(ssd, fn)(**leaf)
        (y[0] if pair else y).sum().backward()
        assert asked[-1] == tuple(n for n in names if n not in frozen)
        for t, n in zip(leaf.values(), names):
            assert (t.grad is None) == (n in frozen)


def test_gradients_that_do_not_exist_are_refused():
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError, match="no gradient 'dy'"):
        ssd.causal_conv_backward(x, torch.zeros(8, 4), gy=x, want=("dx", "dy"))


def test_workspace_queries_do_not_grow_with_the_length():
    """How a sequence is cut is decided in every call: a decision that walks
    along the tokens would delay the launch (0.3 ms at a million of them)."""
    import time
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    lib = _abi.load()
    for L in (1 << 24, 1 << 28, (1 << 31) - 1):
        for b, D in ((8, 5120), (1, 64)):
            d = _abi.SsdScanDims(b, L, D, 16, 1, 1)
            start = time.perf_counter()
            for _ in range(10):
                need = lib.ssd_selective_scan_workspace_size(d, _abi.SSD_BF16)
            assert time.perf_counter() - start < 0.05, (b, L, D)
            assert (need > 0) == (b == 1)


def test_workspaces_are_checked_by_name(monkeypatch):
    """A given workspace that is too small, off its boundary, of another type
    or not dense is refused before the library sees it."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    x, A, B = far(2, 4096, 64), far(64, 16), far(2, 4096, 1, 16)
    need = ssd.selective_scan_workspace_size(x, A, B)
    assert need > 0
    room = far(need + 512, dtype=torch.uint8)
    room = room[-room.data_ptr() % 256:]  # from a boundary on

    def call(workspace):
        ssd.selective_scan_forward(x, x, A, B, B, y=far(2, 4096, 64), workspace=workspace,
                                   return_final_state=False)

    for bad, what in ((room[:need - 1], f"{need - 1} bytes, {need} are needed"),
                      (room[16:], "256 bytes"), (room[::2], "contiguous uint8"),
                      (far(need), "contiguous uint8")):
        with pytest.raises(ValueError, match=f"selective_scan_forward: .*{what}"):
            call(bad)


def test_workspace_sizes_match_the_library():
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    lib = _abi.load()
    x, w = torch.zeros(2, 300, 48), torch.zeros(48, 3)
    d = _abi.SsdConvDims(2, 300, 48, 3, _abi.SSD_ACT_SILU)
    need = lib.ssd_causal_conv_backward_workspace_size(d, _abi.SSD_F32)
    assert ssd.causal_conv_backward_workspace_size(x, w) == need > 0
    A, B = torch.zeros(48, 8), torch.zeros(2, 300, 2, 8)
    d = _abi.SsdScanDims(2, 300, 48, 8, 2, 1)
    need = lib.ssd_selective_scan_backward_workspace_size(d, _abi.SSD_F32)
    assert ssd.selective_scan_backward_workspace_size(x, A, B) == need > 0
    for t, (b, L) in ((x, (2, 300)), (x[0], (1, 300)), (x[:, :1], (1, 2))):
        d = _abi.SsdNormDims(b, L, 48, 3, 1e-5, _abi.SSD_GATE_INPUT, 1)
        need = lib.ssd_gated_norm_backward_workspace_size(d, _abi.SSD_F32)
        assert ssd.gated_norm_backward_workspace_size(t, groups=3) == need > 0
    grads = [torch.zeros(1000), torch.zeros(7, dtype=torch.bfloat16), torch.zeros(0)]
    table = (_abi.SsdGrad * 3)((256, 256, 1000, 0), (512, 512, 7, 1), (0, 0, 0, 0))
    need = lib.ssd_clip_grad_norm_workspace_size(table, 3)
    assert ssd.clip_grad_norm_workspace_size(grads) == need > 0


def test_gate_and_its_values_go_together():
    x, w = torch.zeros(5, 8), torch.zeros(8)
    for gate in ("input", "output"):
        with pytest.raises(ValueError, match=f"gate '{gate}' needs z"):
            ssd.gated_norm_forward(x, w, gate=gate)
        with pytest.raises(ValueError, match=f"gate '{gate}' needs z"):
            ssd.gated_norm_backward(x, w, gy=x, gate=gate)
    with pytest.raises(ValueError, match="gate '.*' needs z"):
        ssd.gated_norm(x, w)  # the default gate
    with pytest.raises(ValueError, match="gate is 'none'"):
        ssd.gated_norm_forward(x, w, z=x, gate="none")


def test_a_workspace_that_is_not_needed_is_not_looked_at(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    x, A, B = far(2, 5, 8), far(8, 4), far(2, 5, 1, 4)
    assert ssd.selective_scan_workspace_size(x, A, B) == 0
    room = far(512, dtype=torch.uint8)
    off = room[-room.data_ptr() % 256 + 16:][:8]
    with pytest.raises(ValueError, match="current device"):  # what is wrong next
        ssd.selective_scan_forward(x, x, A, B, B, y=far(2, 5, 8), workspace=off,
                                   return_final_state=False)


def test_rows_that_share_addresses():
    """The rule for two axes of rows against a count of the addresses."""
    from mamba_ssd_forward_gb300.layer import _apart
    seen = set()
    for b in (1, 2, 3, 5):
        for L in (1, 2, 4):
            for D in (1, 3):
                for bs in range(0, 18):
                    for ts in range(0, 18):
                        t = torch.empty(200).as_strided((b, L, D), (bs, ts, 1))
                        all_of = torch.arange(200).as_strided((b, L, D), (bs, ts, 1)).flatten()
                        want = all_of.unique().numel() == all_of.numel()
                        assert _apart(t) == want, (b, L, D, bs, ts)
                        seen.add((want, bs < ts))
    assert len(seen) == 4


def test_outputs_whose_rows_share_addresses_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    x, w, tok = far(2, 5, 8), far(8, 4), far(2, 8)
    A, B = far(8, 4), far(2, 5, 1, 4)
    for y in (far(5, 8).expand(2, 5, 8), far(2, 1, 8).expand(2, 5, 8), far(1, 8).expand(2, 5, 8),
              far(100).as_strided((2, 5, 8), (40, 4, 1))):
        for call in (lambda: ssd.causal_conv_forward(x, w, y=y),
                     lambda: ssd.selective_scan_forward(x, x, A, B, B, y=y),
                     lambda: ssd.gated_norm_forward(x, far(8), gate="none", y=y)):
            with pytest.raises(ValueError, match="y: rows of an output must not share"):
                call()
    y = far(8).expand(2, 8)
    for call in (lambda: ssd.causal_conv_step(tok, w, None, far(2, 3, 8), y=y),
                 lambda: ssd.selective_scan_step(tok, tok, A, B[:, 0], B[:, 0], None, None, None,
                                                 far(2, 8, 4), y=y),
                 lambda: ssd.gated_norm_forward(tok, far(8), gate="none", y=y)):
        with pytest.raises(ValueError, match="y: rows of an output must not share"):
            call()


def test_the_library_refuses_outputs_whose_rows_share_addresses():
    """Nothing is launched: every call here has a view that is refused."""
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    lib, ok = _abi.load(), 1 << 20
    b, L, D = 3, 8, 64
    x = _abi.SsdSeq(ok, L * D, D)
    conv, one = (_abi.SsdConvDims(b, n, D, 4, 1) for n in (L, 1))
    scan, scan1 = (_abi.SsdScanDims(b, n, D, 16, 2, 1) for n in (L, 1))
    norm = _abi.SsdNormDims(b, L, D, 2, 1e-5, 1, 0)
    ins, big = [x, x, ok, x, x, None, None, None], 1 << 40
    # (batch, token) strides: repeated sequences or tokens, rows half apart, a
    # sequence on another's last rows, one token of one sequence on another's
    for bs, ts in ((0, D), (L * D, 0), (L * D, D - 1), (L * D - 1, D), (D, 2 * D), (3 * D, 2 * D)):
        y = _abi.SsdSeq(ok, bs, ts)
        assert lib.ssd_causal_conv(conv, 1, x, ok, None, None, None, y, None, None) == 1
        assert lib.ssd_causal_conv_backward(conv, 1, x, ok, None, None, x, None, None, y, ok,
                                            None, None, ok, big, None) == 1
        assert lib.ssd_selective_scan(scan, 1, *ins, None, None, y, None, ok, big, None) == 1
        for k in ("du", "ddt", "dB", "dC"):
            v = y if k in ("du", "ddt") else _abi.SsdSeq(ok, bs // 2, ts // 2)  # rows of 32
            g = _abi.SsdScanGrads(**{**dict(du=x, ddt=x, dB=x, dC=x), k: v})
            assert lib.ssd_selective_scan_backward(scan, 1, *ins, None, x, None, None, g, ok,
                                                   big, None) == 1, k
        assert lib.ssd_gated_norm(norm, 1, x, ok, None, x, y, None) == 1
        for dx, dz in ((x, y), (y, x)):
            assert lib.ssd_gated_norm_backward(norm, 1, x, ok, None, x, x, dx, dz, ok, None, ok,
                                               big, None) == 1
    y = _abi.SsdSeq(ok, D - 1, 0)
    assert lib.ssd_causal_conv_step(one, 1, x, ok, None, ok, y, None) == 1
    assert lib.ssd_selective_scan_step(scan1, 1, *ins, ok, y, None) == 1


def test_norm_takes_as_many_sequences_as_tokens():
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    lib = _abi.load()

    def need(b, L):
        d = _abi.SsdNormDims(b, L, 64, 2, 1e-5, 1, 0)
        return lib.ssd_gated_norm_backward_workspace_size(d, 1)

    assert need(1 << 17, 3) == need(1, 3 << 17) > 0
    assert need(65536, 1) > 0 and need((1 << 31) - 1, 1) > 0
    assert need(1 << 16, 1 << 15) == 0  # 2^31 tokens


def test_outputs_in_memory_that_is_still_read_are_refused(monkeypatch):
    """Threads of the same launch read the convolution's tokens in front of
    theirs, and h0 at the start of every segment."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    x, w, h = far(2, 5, 8), far(8, 4), far(2, 8, 4)
    A, B = far(8, 4), far(2, 5, 1, 4)
    with pytest.raises(ValueError, match="y must not be the memory of x"):
        ssd.causal_conv_forward(x, w, y=x)
    with pytest.raises(ValueError, match="final_state must not be the memory of h0"):
        ssd.selective_scan_forward(x, x, A, B, B, h0=h, final_state=h, y=far(2, 5, 8))
    from mamba_ssd_forward_gb300 import _abi, build
    build.build()
    lib, ok = _abi.load(), 1 << 20
    v, y = _abi.SsdSeq(ok, 512, 64), _abi.SsdSeq(2 * ok, 512, 64)
    conv = _abi.SsdConvDims(2, 8, 64, 4, 1)
    assert lib.ssd_causal_conv(conv, 1, v, ok, None, None, None, v, None, None) == 1
    scan = _abi.SsdScanDims(2, 8, 64, 16, 2, 1)
    assert lib.ssd_selective_scan(scan, 1, v, v, ok, v, v, None, None, None, ok, None, y, ok, ok,
                                  1 << 40, None) == 1


def test_a_gradient_given_twice_is_refused():
    t, e = far(10), far(0)
    with pytest.raises(ValueError, match="more than once"):
        ssd.clip_grad_norm([t, far(3), t], 1.0)
    with pytest.raises(ValueError, match="more than once"):
        ssd.clip_grad_norm([far(10), far(10)], 1.0, out=[t, t])
    with pytest.raises(Exception) as other:  # empty ones may be: there is no such device
        ssd.clip_grad_norm([e, t, e], 1.0)
    assert "more than once" not in str(other.value)
