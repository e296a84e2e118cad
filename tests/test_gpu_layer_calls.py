"""How the operators around the scan are called: from several host threads, in
graphs, with some gradients only, with given outputs and workspaces, and with
values at the ends of the number range."""
import threading

import pytest
import torch

from layer_cases import conv_inputs, lengths_of, norm_inputs, scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_forward_gb300 import build
    build.build()
    import mamba_ssd_forward_gb300 as m
    return m


def test_norms_of_two_widths_from_two_threads(ssd):
    """Groups of 8192 and of 512 channels run the same kernel with different
    amounts of shared memory; neither call may undo the other's."""
    from mamba_ssd_forward_gb300 import _abi
    lib, calls, kept = _abi.load(), [], []
    for D in (8192, 512):
        a, gy = norm_inputs(2, D, "bf16", bias=False)
        d = _abi.SsdNormDims(1, 2, D, 1, 1e-5, _abi.SSD_GATE_INPUT, 0)
        ws = torch.empty(lib.ssd_gated_norm_backward_workspace_size(d, _abi.SSD_BF16),
                         dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(a["x"]) for _ in range(3)]
        dw = torch.empty_like(a["weight"])
        x, z, g, y, dx, dz = (_abi.SsdSeq(t.data_ptr(), 0, D) for t in (a["x"], a["z"], gy, *outs))
        w, st = a["weight"].data_ptr(), torch.cuda.Stream()
        kept += [a, gy, ws, outs, dw, st]
        calls.append((
            (d, _abi.SSD_BF16, x, w, None, z, y, st.cuda_stream),
            (d, _abi.SSD_BF16, x, w, None, z, g, dx, dz, dw.data_ptr(), None, ws.data_ptr(),
             ws.numel(), st.cuda_stream)))
    torch.cuda.synchronize()
    start, codes = threading.Barrier(2), [set(), set()]

    def work(k):
        forward, backward = calls[k]
        start.wait()
        for _ in range(10000):  # the library runs without the interpreter's lock
            codes[k].add(lib.ssd_gated_norm(*forward))
            codes[k].add(lib.ssd_gated_norm_backward(*backward))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}, {0}]


def test_norms_of_two_widths_in_one_graph(ssd):
    cases = [norm_inputs(3, D, "bf16", seed=D, bias=False) for D in (8192, 512)]

    def everything():
        out = []
        for a, gy in cases:
            out += [ssd.gated_norm_forward(**a), ssd.gated_norm_backward(**a, gy=gy)["dx"]]
        return out

    ref = [t.clone() for t in everything()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, got))


def test_first_derivatives_within_a_graph_and_no_second(ssd):
    a, gy, _ = conv_inputs(2, 20, 24, 4, "fp32", seed=3)
    leaf = {k: v.clone().requires_grad_() for k, v in a.items()}
    y = ssd.causal_conv(**leaf)[0]
    g = torch.autograd.grad(y, list(leaf.values()), gy, create_graph=True)
    ref = ssd.causal_conv_backward(**a, gy=gy)
    for k, got in zip(leaf, g):
        assert torch.equal(got, ref["d" + k]), k
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad((g[0] ** 2).sum(), leaf["x"])


def test_some_gradients_only(ssd):
    """Those asked for have the same bits; the others are None."""
    a, gy, gf = conv_inputs(2, 40, 24, 4, "bf16", seed=3)
    s, sgy, sgf = scan_inputs(2, 40, 24, 16, 1, "bf16", seed=3)
    n, ngy = norm_inputs(30, 24, "bf16", seed=3)
    for fn, args, more, always in (
            (ssd.causal_conv_backward, a, dict(gy=gy, gfinal=gf), ()),
            (ssd.selective_scan_backward, s, dict(gy=sgy, gfinal=sgf, dt_softplus=True),
             ("du", "ddt", "dB", "dC")),
            (ssd.gated_norm_backward, n, dict(gy=ngy), ("dx", "dz"))):
        full = fn(**args, **more)
        assert all(v is not None for v in full.values())
        for want in [()] + [(k,) for k in full] + [tuple(full)]:
            got = fn(**args, **more, want=want)
            assert got.keys() == full.keys()
            for k, v in got.items():
                assert (v is not None) == (k in want or k in always), (want, k)
                assert v is None or torch.equal(v, full[k]), (want, k)
    ssd.device_error()


# aligned and not: the schedules, and what they keep in the workspace, differ
@pytest.mark.parametrize("wide", [0, 1])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_given_workspaces(ssd, dtype, wide):
    """Workspaces of the queried sizes, not initialised and nothing behind
    them: the same bits, and the bytes behind them stay."""
    a, gy, gf = conv_inputs(3, 700, 132, 4, dtype, seed=5, wide=wide)
    s, sgy, sgf = scan_inputs(3, 700, 132, 16, 2, dtype, seed=5, wide=wide)
    n, ngy = norm_inputs(900, 264, dtype, seed=5, wide=wide)
    big, gbig = norm_inputs(5, 20480, dtype, seed=6, wide=wide)
    grads = [torch.randn(300000, device="cuda"), torch.randn(77, device="cuda").bfloat16()]
    scaled = [torch.empty_like(t) for t in grads]
    calls = [
        (ssd.causal_conv_backward, dict(a, gy=gy, gfinal=gf),
         ssd.causal_conv_backward_workspace_size(a["x"], a["weight"])),
        (ssd.selective_scan_forward, dict(s, dt_softplus=True),
         ssd.selective_scan_workspace_size(s["u"], s["A"], s["B"])),
        (ssd.selective_scan_backward, dict(s, gy=sgy, gfinal=sgf, dt_softplus=True),
         ssd.selective_scan_backward_workspace_size(s["u"], s["A"], s["B"])),
        (ssd.gated_norm_backward, dict(n, gy=ngy, groups=2),
         ssd.gated_norm_backward_workspace_size(n["x"], groups=2)),
        (ssd.gated_norm_backward, dict(big, gy=gbig),
         ssd.gated_norm_backward_workspace_size(big["x"])),
        (ssd.clip_grad_norm, dict(grads=grads, max_norm=0.5, out=scaled),
         ssd.clip_grad_norm_workspace_size(grads)),
    ]
    for fn, args, need in calls:
        assert need > 0, fn

        def outputs(r):
            r = list(r.values()) if isinstance(r, dict) else [r] if torch.is_tensor(r) else list(r)
            return [t.clone() for t in r + (scaled if fn is ssd.clip_grad_norm else [])]

        ref = outputs(fn(**args))
        room = torch.full((need + 65536,), 255, dtype=torch.uint8, device="cuda")  # NaN
        got = outputs(fn(**args, workspace=room[:need]))
        assert all(torch.equal(p, q) for p, q in zip(ref, got)), fn
        assert bool((room[need:] == 255).all()), fn
    ssd.device_error()


def test_outputs_of_any_order_of_rows(ssd):
    """Tokens before sequences, and rows of two sequences between each other."""
    b, L, D = 2, 9, 24
    a, _, _ = conv_inputs(b, L, D, 4, "bf16", seed=8)
    s, _, _ = scan_inputs(b, L, D, 16, 1, "bf16", seed=8)
    n, _ = norm_inputs((b, L), D, "bf16", seed=8)
    for strides in ((D, b * D), (D, 2 * D), (3 * D, 2 * D), (2 * L * D, 2 * D + 1)):
        buf = torch.zeros(4 * L * D + 64, dtype=torch.bfloat16, device="cuda")
        y = buf.as_strided((b, L, D), (*strides, 1))
        for fn, args in ((ssd.causal_conv_forward, a),
                         (ssd.selective_scan_forward, dict(s, dt_softplus=True)),
                         (ssd.gated_norm_forward, n)):
            ref = fn(**args)
            got = fn(**args, y=y)
            if isinstance(ref, tuple):
                ref, got = ref[0], got[0]
            assert got is y and torch.equal(got, ref), (fn, strides)
    ssd.device_error()


# channels of a group that a block's registers hold, and that they do not
@pytest.mark.parametrize("D", [8, 4104])
def test_norm_of_many_sequences(ssd, D):
    """More sequences than a grid's second dimension: as one sequence of all
    their tokens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    b, L = 65537, 2
    x, z, gy = (torch.randn(b, L, D, generator=g, device="cuda") for _ in range(3))
    w = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
    flat = [t.view(1, b * L, D) for t in (x, z, gy)]
    y = ssd.gated_norm_forward(x, w, z=z)
    assert torch.equal(y.view(1, b * L, D), ssd.gated_norm_forward(flat[0], w, z=flat[1]))
    last = ssd.gated_norm_forward(x[-1], w, z=z[-1])
    assert torch.equal(y[-1], last)
    got = ssd.gated_norm_backward(x, w, z=z, gy=gy)
    ref = ssd.gated_norm_backward(flat[0], w, z=flat[1], gy=flat[2])
    for k in ("dx", "dz", "dweight"):
        assert torch.equal(got[k].flatten(), ref[k].flatten()), k
    ssd.device_error()


# within a tile, over several, cut into segments, with sequences that end early
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("b,L,D,N,lengths", [(1, 5, 40, 16, None), (2, 70, 33, 5, [70, 41]),
                                             (2, 700, 64, 16, [700, 333]),
                                             (3, 40, 8, 40, [40, 0, 1])])
def test_states_that_are_forgotten_at_once(ssd, b, L, D, N, lengths, dtype):
    """A = -inf is a decay of zero: as a finite A that is as steep, also where
    the places after a sequence's end hold steps of zero."""
    s, gy, gfinal = scan_inputs(b, L, D, N, 1, dtype, seed=L)
    steep, none = (s["A"].clone() for _ in range(2))
    some = torch.rand(D, N, device="cuda") < 0.3
    some[0, 0], some[-1, -1] = True, True
    steep[some], none[some] = -1e30, -float("inf")
    n = lengths_of(lengths)

    def everything(A):
        a = {**s, "A": A}
        out = list(ssd.selective_scan_forward(**a, lengths=n, dt_softplus=True))
        out += ssd.selective_scan_backward(**a, gy=gy, gfinal=gfinal, lengths=n,
                                           dt_softplus=True).values()
        state = s["h0"].clone()
        at = {k: v[:, 0] if k in ("u", "dt", "B", "C", "z") else v for k, v in a.items()}
        del at["h0"]
        return out + [ssd.selective_scan_step(**at, state=state, dt_softplus=True), state]

    for i, (p, q) in enumerate(zip(everything(steep), everything(none))):
        assert torch.isfinite(p).all() and torch.equal(p, q), i
    ssd.device_error()
