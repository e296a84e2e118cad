"""How the operators around a language model's blocks are called: under autograd, in
graphs, on two streams and from two threads, with given workspaces, some gradients
only, and together in a training step."""
import os
import sys
import threading

import pytest
import torch
import torch.nn.functional as F

import model_ref64 as R

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_forward_gb300 import build
    build.build()
    import mamba_ssd_forward_gb300 as m
    return m


def inputs(seed=0, rows=70, d=64, V=300, io=B16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t = torch.randint(0, V, (rows,), generator=g, device="cuda")
    t[::3] = -100
    return {"x": n(rows, d).to(io), "r": n(rows, d), "w": 1 + 0.2 * n(d), "W": (0.3 * n(V, d)).to(io),
            "t": t, "gy": n(rows, d).to(io), "G": n(96, d).to(io),
            "H": n(40, 2500).to(io)}


def everything(ssd, a):
    y, total = ssd.add_norm_forward(a["x"], a["r"], a["w"])
    g = ssd.add_norm_backward(total, a["w"], a["gy"], a["r"])
    q, s, _ = ssd.add_norm_quantized(a["x"], a["r"], a["w"], block=32)
    loss, lse = ssd.linear_cross_entropy_forward(y, a["W"], a["t"], reduction="mean")
    b = ssd.linear_cross_entropy_backward(y, a["W"], a["t"], lse, loss, reduction="mean")
    return [y, total, *g.values(), q.float(), s, loss, lse, *b.values(),
            *(ssd.orthogonalize(a[k], dtype=to) for k in "GH" for to in (B16, F32))]


@pytest.mark.parametrize("io", [B16, F32], ids=str)
def test_calls_repeat_bit_for_bit(ssd, io):
    a = inputs(1, 500, 200, 3000, io)
    for p, q in zip(everything(ssd, a), everything(ssd, a)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("io", [B16, F32], ids=str)
def test_captured_and_replayed_on_new_inputs(ssd, io):
    a, b = inputs(1, io=io), inputs(2, io=io)
    b["t"][:] = -100  # fewer tokens with a target than when it was captured: one
    b["t"][5] = 7
    everything(ssd, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(ssd, a)
    for c in (b, inputs(3, io=io)):
        for k in a:
            a[k].copy_(c[k])
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, everything(ssd, c)):
            assert torch.equal(p, q)


def test_two_graphs_on_two_streams(ssd):
    """Each with its own workspaces, replayed together."""
    ins, graphs, outs, streams = [inputs(i, 300, 128, 2000) for i in (1, 2)], [], [], []
    refs = [[t.clone() for t in everything(ssd, a)] for a in ins]
    for a in ins:
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            outs.append(everything(ssd, a))
        graphs.append(g)
        streams.append(s)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, refs):
        for p, q in zip(got, ref):
            assert torch.equal(p, q)


def test_two_threads(ssd):
    ins = [inputs(1, 300, 128, 2000), inputs(2, 45, 72, 900)]
    refs = [[t.clone() for t in everything(ssd, a)] for a in ins]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(2)

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for _ in range(20):
                got = everything(ssd, ins[k])
                torch.cuda.current_stream().synchronize()
                bad.extend(i for i, (p, q) in enumerate(zip(got, refs[k])) if not torch.equal(p, q))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("io", [B16, F32], ids=str)
def test_workspaces_of_the_callers(ssd, io):
    """Of the size that is asked for, whatever they hold, with nothing written behind."""
    a = inputs(4, 130, 80, 700, io)
    y, total = ssd.add_norm_forward(a["x"], a["r"], a["w"])
    lse = ssd.linear_cross_entropy_forward(y, a["W"], a["t"])[1]
    calls = [
        (ssd.add_norm_backward_workspace_size(total, a["gy"]),
         lambda **k: list(ssd.add_norm_backward(total, a["w"], a["gy"], **k).values())),
        (ssd.linear_cross_entropy_workspace_size(y, a["W"]),
         lambda **k: list(ssd.linear_cross_entropy_forward(y, a["W"], a["t"], **k))),
        (ssd.linear_cross_entropy_backward_workspace_size(y, a["W"]),
         lambda **k: list(ssd.linear_cross_entropy_backward(y, a["W"], a["t"], lse, **k).values())),
        (ssd.orthogonalize_workspace_size(a["G"]), lambda **k: [ssd.orthogonalize(a["G"], **k)]),
        (ssd.orthogonalize_workspace_size(a["G"], F32),
         lambda **k: [ssd.orthogonalize(a["G"], dtype=F32, **k)]),
        (ssd.orthogonalize_workspace_size(a["H"], F32),
         lambda **k: [ssd.orthogonalize(a["H"], dtype=F32, **k)])]
    for need, call in calls:
        ref = call()
        for fill in (0xff, 0x7f, 0):
            ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
            for p, q in zip(call(workspace=ws[:need]), ref):
                assert torch.equal(p, q)
            assert (ws[need:] == fill).all()
        with pytest.raises(ValueError, match="are needed"):
            call(workspace=ws[:need - 1])


def test_some_gradients_only(ssd):
    a = inputs(5)
    y, total = ssd.add_norm_forward(a["x"], a["r"], a["w"])
    lse = ssd.linear_cross_entropy_forward(y, a["W"], a["t"])[1]
    for fn in (lambda w: ssd.add_norm_backward(total, a["w"], a["gy"], want=w),
               lambda w: ssd.linear_cross_entropy_backward(y, a["W"], a["t"], lse, want=w)):
        full = fn(None)
        assert all(v is not None for v in full.values())
        for want in [()] + [(k,) for k in full] + [tuple(full)]:
            got = fn(want)
            for k, v in got.items():
                assert (v is None) if k not in want else torch.equal(v, full[k]), (want, k)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_autograd_gives_the_backward_calls(ssd, reduction):
    a = inputs(6)
    leaf = {k: a[k].clone().requires_grad_() for k in ("x", "r", "w", "W")}
    y, total = ssd.add_norm(leaf["x"], leaf["r"], leaf["w"])
    loss = ssd.linear_cross_entropy(y, leaf["W"], a["t"], reduction=reduction)
    out = loss.sum() * 3 + (total * a["r"]).sum()
    got = torch.autograd.grad(out, list(leaf.values()))
    with torch.no_grad():
        y, total = ssd.add_norm_forward(a["x"], a["r"], a["w"])
        _, lse = ssd.linear_cross_entropy_forward(y, a["W"], a["t"])
        gloss = torch.full(loss.shape, 3.0, device="cuda")
        b = ssd.linear_cross_entropy_backward(y, a["W"], a["t"], lse, gloss, reduction=reduction)
        g = ssd.add_norm_backward(total, a["w"], b["dx"], a["r"])
    for p, q in zip(got, (g["dx"], g["dresidual"], g["dweight"], b["dweight"])):
        assert torch.equal(p, q)


@pytest.mark.parametrize("used", ["y", "total"])
def test_autograd_of_one_output(ssd, used):
    """What nothing uses has no gradient: that of zeros."""
    a = inputs(12)
    leaf = {k: a[k].clone().requires_grad_() for k in ("x", "r", "w")}
    y, total = ssd.add_norm(*leaf.values())
    zero = torch.zeros_like
    out, gy, gt = (y, a["gy"], zero(total)) if used == "y" else (total, zero(y), a["r"])
    got = torch.autograd.grad(out, list(leaf.values()), gy if used == "y" else gt)
    ref = ssd.add_norm_backward(total.detach(), a["w"], gy, gt)
    for p, k in zip(got, ("dx", "dresidual", "dweight")):
        assert torch.equal(p, ref[k]), k


def test_no_second_derivatives(ssd):
    a = inputs(7, io=F32)
    x = a["x"].requires_grad_()
    loss = ssd.linear_cross_entropy(x, a["W"], a["t"])
    g = torch.autograd.grad(loss, x, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad((g ** 2).sum(), x)
    y, _ = ssd.add_norm(x, a["r"], a["w"])
    g = torch.autograd.grad(y.sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad((g ** 2).sum(), x)


def test_broadcast_gradients_and_inputs(ssd):
    """Cotangents that autograd expands, one row of hidden states for all tokens, and a
    residual shared by two blocks."""
    a = inputs(8, io=F32)
    row = a["x"][:1].clone().requires_grad_()
    W = a["W"].clone().requires_grad_()
    loss = ssd.linear_cross_entropy(row.expand(70, -1), W, a["t"], reduction="sum")
    drow, dW = torch.autograd.grad(loss, (row, W))
    live = int((a["t"] >= 0).sum())
    z = (row.detach() @ W.detach().t()).double()
    p = torch.softmax(z, 1)[0]
    count = torch.bincount(a["t"][a["t"] >= 0], minlength=300).double()
    ref = (live * p - count) @ W.detach().double()
    assert float((drow[0].double() - ref).norm() / ref.norm()) < 1e-4
    r = a["r"].clone().requires_grad_()
    y1, t1 = ssd.add_norm(a["x"], r, a["w"])
    y2, t2 = ssd.add_norm(y1, t1, a["w"])
    got = torch.autograd.grad(y2.sum() + t2.mean(), r)[0]
    rd = a["r"].double().requires_grad_()
    u1, v1 = R.add_norm(a["x"], rd, a["w"])
    u2, v2 = R.add_norm(u1, v1, a["w"])
    ref = torch.autograd.grad(u2.sum() + v2.mean(), rd)[0]
    assert float((got.double() - ref).norm() / ref.norm()) < 1e-4


def test_capture_of_a_training_step(ssd):
    """Forward and backward captured together, while nothing else of the leaves lives."""
    a = inputs(9)
    x = a["x"].clone().requires_grad_()
    W = a["W"].clone().requires_grad_()

    def step():
        y, total = ssd.add_norm(x, a["r"], a["w"])
        loss = ssd.linear_cross_entropy(y, W, a["t"])
        return (loss.detach(), *torch.autograd.grad(loss, (x, W)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ref = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, ref):
        assert torch.equal(p, q)


def test_the_example_runs_and_its_gradients_hold(ssd):
    """examples/language_model.py: a model of blocks with these operators around them; its
    gradients against the same model with the operators' definitions in torch."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import language_model as M
    torch.manual_seed(0)
    model = M.Model(words=500, width=128)
    tokens = torch.randint(0, 500, (2, 65), device="cuda")
    tokens[1, 40:] = -100  # a shorter document
    loss = model.loss(tokens)
    params = list(model.p.values())
    got = torch.autograd.grad(loss, params)

    def norm(x, r, w):
        t = x.float() + r
        y = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-5) * w
        return y.to(x.dtype), t

    def entropy(x, W, t, reduction):
        z = x.float().flatten(0, 1) @ W.float().t()
        return F.cross_entropy(z, t.flatten(), ignore_index=-100, reduction=reduction)

    ref_loss = model.loss(tokens, norm=norm, entropy=entropy)
    ref = torch.autograd.grad(ref_loss, params)
    assert abs(float(loss.detach() - ref_loss.detach())) < 1e-2 * float(ref_loss.detach())
    for k, g, h in zip(model.p, got, ref):
        g, h = g.double(), h.double()
        # bf16 activations and gradients through two blocks: some eight roundings of 2^-9
        assert float((g - h).norm() / h.norm()) < 0.03, k
    assert len(M.train(model, tokens, steps=2)) == 2
    out = M.serve(model, tokens[:, :8].clamp(min=0), new=3)
    assert out.shape == (2, 3) and bool((out >= 0).all()) and bool((out < 500).all())
