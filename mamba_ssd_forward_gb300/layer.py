"""The operators around a state space scan in a layer (include/ssd_layer.h):
the short causal convolution, the selective scan, the gated group norm and
the global gradient norm with clipping.

As in the rest of the package, the functions here check types and shapes,
allocate outputs and workspaces on the current CUDA stream and pass pointers;
all arithmetic runs in the library's kernels.

Activations ([b, L, D] and the like) may be views with any strides between
sequences and tokens as long as the last axis is dense, such as slices of a
wider projection; other views are refused.  `lengths` (int32 [b] on the
device, or None) gives the real tokens of each padded sequence.  The tensors'
device has to be the current one.
"""
from __future__ import annotations

import functools
import struct

import torch

from . import _abi
from ._abi import SsdSeq

_GATES = {"none": _abi.SSD_GATE_NONE, "input": _abi.SSD_GATE_INPUT,
          "output": _abi.SSD_GATE_OUTPUT}
_ACTS = {None: _abi.SSD_ACT_NONE, "silu": _abi.SSD_ACT_SILU}
_IO = {torch.float32: _abi.SSD_F32, torch.bfloat16: _abi.SSD_BF16}


def _io(t, name):
    try:
        return _IO[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}") from None


def _stream(like):
    """The current stream.  The library launches on the current device, which
    therefore has to be the tensor's."""
    dev = like.get_device()
    if dev != (current := torch._C._cuda_getDevice()):
        raise ValueError(f"the tensors are on cuda:{dev} but the current device is "
                         f"cuda:{current}: call within torch.cuda.device({dev})")
    return torch._C._cuda_getCurrentRawStream(dev)


def _refuse(t, name, shape, dtype, like):
    """Says what is wrong with a tensor that is not as it has to be."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a CUDA tensor on the same device as the input")
    raise ValueError(f"{name} must be contiguous" if t.stride()[-1:] == (1,) else
                     f"{name} must be dense along its last axes")


def _dense(t, name, shape, dtype, like):
    """Address of a dense tensor (None stays None)."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or (dev := t.get_device()) < 0 or dev != like.get_device()):
        _refuse(t, name, shape, dtype, like)
    return t.data_ptr()


def _seq(t, name, shape, dtype, like):
    """View of an activation [b, L, D]; None stays None."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or (dev := t.get_device()) < 0
            or dev != like.get_device()):
        _refuse(t, name, shape, dtype, like)
    sb, st, sc = t.stride()
    if sc != 1 and shape[2] != 1:
        _refuse(t, name, shape, dtype, like)
    return SsdSeq(t.data_ptr(), sb if shape[0] > 1 else 0, st if shape[1] > 1 else 0)


def _token(t, name, shape, dtype, like):
    """The same of one token each, [b, D]."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or (dev := t.get_device()) < 0
            or dev != like.get_device()):
        _refuse(t, name, shape, dtype, like)
    sb, sc = t.stride()
    if sc != 1 and shape[1] != 1:
        _refuse(t, name, shape, dtype, like)
    return SsdSeq(t.data_ptr(), sb if shape[0] > 1 else 0, 0)


def _grouped(t, name, shape, dtype, like):
    """A view [b, L, G, N] or [b, G, N] whose last two axes are dense together."""
    if (t.dtype is not dtype or t.shape != shape or (dev := t.get_device()) < 0
            or dev != like.get_device()):
        _refuse(t, name, shape, dtype, like)
    *lead, sg, sn = t.stride()
    if (sn != 1 and shape[-1] != 1) or (sg != shape[-1] and shape[-2] != 1):
        raise ValueError(f"{name} must be dense along its last axes")
    return SsdSeq(t.data_ptr(), lead[0] if shape[0] > 1 else 0,
                  lead[1] if len(lead) == 2 and shape[1] > 1 else 0)


def _sized(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _workspace(need, workspace, like, fn):
    """(tensor kept alive, address, bytes) of a workspace of `need` bytes."""
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = _sized(need, like.device)
        return workspace, workspace.data_ptr(), need
    if (workspace.dtype != torch.uint8 or workspace.device != like.device
            or not workspace.is_contiguous()):
        raise ValueError(f"{fn}: workspace must be a contiguous uint8 tensor on the inputs' device")
    at, have = workspace.data_ptr(), workspace.numel()
    if have < need:
        raise ValueError(f"{fn}: workspace has {have} bytes, {need} are needed")
    if at % 256:
        raise ValueError(f"{fn}: workspace must start on 256 bytes")
    return workspace, at, have


def _lengths(lengths, b, like):
    return _dense(lengths, "lengths", (b,), torch.int32, like)


def _out(t, name, shape, dtype, like):
    """A given output, whose rows have to lie apart, or a new dense one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if t.shape == shape and not t.is_contiguous() and not _apart(t):
        raise ValueError(f"{name}: rows of an output must not share addresses "
                         f"(strides {t.stride()} for {tuple(shape)})")
    return t


def _separate(out, name, source, source_name):
    """Refuses an output given in the memory of an input that other threads
    still read."""
    if out is not None and source is not None and out.data_ptr() == source.data_ptr():
        raise ValueError(f"{name} must not be the memory of {source_name}")


def _apart(t):
    """Whether the rows [.., D] of a view of two or three axes lie apart."""
    *sizes, D = t.shape
    steps = [(s, n) for s, n in zip(t.stride(), sizes) if n > 1]
    if any(s < D for s, _ in steps):
        return False
    if len(steps) < 2:
        return True
    (s, n), (large, m) = sorted(steps)
    # rows k large steps apart against those j, j + 1 small ones apart
    return large >= (n - 1) * s + D or all(
        k * large // s >= n or (k * large % s >= D and
                                (k * large // s + 1 >= n or s - k * large % s >= D))
        for k in range(1, m))


class _Last(torch.autograd.Function):
    """A gradient that stands for a function of `sources` without a gradient
    of its own: differentiating it raises."""

    @staticmethod
    def forward(ctx, grad, *sources):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("second derivatives of this library's operators are not available")


def _wanted(want, names, fn):
    """The gradients asked for: a function of the name and of whether the
    input is there."""
    if want is None:
        return lambda name, there=True: there
    if unknown := set(want) - set(names):
        raise ValueError(f"{fn}: no gradient {sorted(unknown)[0]!r} (there are {', '.join(names)})")
    return lambda name, there=True: there and name in want


def _needed(ctx, names):
    """The gradients that autograd asks for, by the leading inputs' names."""
    return tuple(n for n, need in zip(names, ctx.needs_input_grad) if need)


def _first_order(backward):
    """Wraps the backward pass of an autograd function whose gradients come
    from kernels, which autograd cannot follow.  Under create_graph they would
    come back as constants and a term that depends on them lose its part
    silently."""
    @functools.wraps(backward)
    def wrapped(ctx, *cotangents):
        if not torch.is_grad_enabled():
            return backward(ctx, *cotangents)
        with torch.no_grad():
            grads = backward(ctx, *cotangents)
        sources = [t for t in (*ctx.saved_tensors, *cotangents)
                   if t is not None and t.requires_grad]
        return tuple(None if g is None else _Last.apply(g, *sources) for g in grads)
    return wrapped


# ------------------------------------------------------ causal convolution

def _conv_dims(x, weight, activation, step=False):
    if activation not in _ACTS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    if x.dim() != (2 if step else 3) or weight.dim() != 2:
        raise ValueError("x must be [b, D] and weight [D, W]" if step else
                         "x must be [b, L, D] and weight [D, W]")
    b, D = x.shape[0], x.shape[-1]
    return _abi.SsdConvDims(b, 1 if step else x.shape[1], D, weight.shape[1], _ACTS[activation])


def causal_conv_forward(x, weight, bias=None, state=None, lengths=None, activation="silu",
                        y=None, final_state=None, return_final_state: bool = True):
    """y [b, L, D], final_state [b, W - 1, D] = the causal convolution of each
    channel with its W (2 to 4) weights and SiLU (ssd_causal_conv).

    x [b, L, D] and state [b, W - 1, D] (the inputs before the first token,
    oldest first; None = zeros) in the I/O type, weight [D, W] and bias [D]
    float32.  final_state holds the last W - 1 inputs, for a later call or
    causal_conv_step.  y must not be x."""
    d = _conv_dims(x, weight, activation)
    _separate(y, "y", x, "x")
    io, b, L, D, W = _io(x, "x"), d.batch, d.seqlen, d.channels, d.width
    y = _out(y, "y", (b, L, D), x.dtype, x)
    keep = (b, W - 1, D)
    if final_state is None and return_final_state:
        final_state = torch.empty(keep, dtype=x.dtype, device=x.device)
    _abi.check("ssd_causal_conv", _abi.load().ssd_causal_conv(
        d, io, _seq(x, "x", (b, L, D), x.dtype, x),
        _dense(weight, "weight", (D, W), torch.float32, x),
        _dense(bias, "bias", (D,), torch.float32, x), _dense(state, "state", keep, x.dtype, x),
        _lengths(lengths, b, x), _seq(y, "y", (b, L, D), x.dtype, x),
        _dense(final_state, "final_state", keep, x.dtype, x), _stream(x)))
    return y, final_state


_CONV_GRADS = ("dx", "dweight", "dbias", "dstate")


def causal_conv_backward_workspace_size(x, weight) -> int:
    """Bytes of workspace that causal_conv_backward needs."""
    d = _conv_dims(x, weight, None)
    return int(_abi.load().ssd_causal_conv_backward_workspace_size(d, _io(x, "x")))


def causal_conv_backward(x, weight, bias=None, state=None, gy=None, gfinal=None, lengths=None,
                         activation="silu", workspace=None, want=None) -> dict:
    """Gradients through causal_conv_forward given gy = dL/dy and gfinal =
    dL/dfinal_state (None = 0), by ssd_causal_conv_backward: a dict of dx (I/O
    type), dweight, dbias (float32; dbias None without a bias) and dstate (None
    without a state).  `want` names those to compute (None = all); the others
    are None."""
    if gy is None:
        raise ValueError("gy (dL/dy) is required")
    has = _wanted(want, _CONV_GRADS, "causal_conv_backward")
    d = _conv_dims(x, weight, activation)
    io, b, L, D, W = _io(x, "x"), d.batch, d.seqlen, d.channels, d.width
    lib, keep = _abi.load(), (b, W - 1, D)
    ws, wp, wn = _workspace(lib.ssd_causal_conv_backward_workspace_size(d, io), workspace, x,
                            "causal_conv_backward")

    def out(name, there, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=x.device) if has(name, there) else None

    dx = out("dx", True, (b, L, D), x.dtype)
    dw = out("dweight", True, (D, W), torch.float32)
    db = out("dbias", bias is not None, (D,), torch.float32)
    ds = out("dstate", state is not None, keep, x.dtype)
    _abi.check("ssd_causal_conv_backward", lib.ssd_causal_conv_backward(
        d, io, _seq(x, "x", (b, L, D), x.dtype, x),
        _dense(weight, "weight", (D, W), torch.float32, x),
        _dense(bias, "bias", (D,), torch.float32, x), _dense(state, "state", keep, x.dtype, x),
        _seq(gy, "gy", (b, L, D), x.dtype, x), _dense(gfinal, "gfinal", keep, x.dtype, x),
        _lengths(lengths, b, x), _seq(dx, "dx", (b, L, D), x.dtype, x),
        *(None if t is None else t.data_ptr() for t in (dw, db, ds)), wp, wn, _stream(x)))
    return {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds}


def causal_conv_step(x, weight, bias, state, activation="silu", y=None):
    """y [b, D] = one token of the convolution for every sequence
    (ssd_causal_conv_step).  state [b, W - 1, D] is updated in place."""
    d = _conv_dims(x, weight, activation, step=True)
    b, D, W = d.batch, d.channels, d.width
    y = _out(y, "y", (b, D), x.dtype, x)
    if state is None:
        raise ValueError("state is required")
    _abi.check("ssd_causal_conv_step", _abi.load().ssd_causal_conv_step(
        d, _io(x, "x"), _token(x, "x", (b, D), x.dtype, x),
        _dense(weight, "weight", (D, W), torch.float32, x),
        _dense(bias, "bias", (D,), torch.float32, x),
        _dense(state, "state", (b, W - 1, D), x.dtype, x), _token(y, "y", (b, D), x.dtype, x),
        _stream(x)))
    return y


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, lengths, activation):
        y, final_state = causal_conv_forward(x, weight, bias, state, lengths, activation)
        ctx.save_for_backward(x, weight, bias, state, lengths)
        ctx.activation = activation
        return y, final_state

    @staticmethod
    @_first_order
    def backward(ctx, gy, gfinal):
        x, weight, bias, state, lengths = ctx.saved_tensors
        g = causal_conv_backward(x, weight, bias, state, gy.contiguous(), gfinal.contiguous(),
                                 lengths, ctx.activation, want=_needed(ctx, _CONV_GRADS))
        return (*(g[k] for k in _CONV_GRADS), None, None)


def causal_conv(x, weight, bias=None, state=None, lengths=None, activation="silu"):
    """y, final_state = causal_conv_forward, differentiable with respect to x,
    weight, bias and state."""
    return _CausalConv.apply(x, weight, bias, state, lengths, activation)


# ----------------------------------------------------------- selective scan

def _scan_dims(u, A, B, dt_softplus, step=False):
    if u.dim() != (2 if step else 3) or A.dim() != 2 or B.dim() != u.dim() + 1:
        raise ValueError("u must be [b, D], A [D, N] and B, C [b, G, N]" if step else
                         "u must be [b, L, D], A [D, N] and B, C [b, L, G, N]")
    b, D = u.shape[0], u.shape[-1]
    return _abi.SsdScanDims(b, 1 if step else u.shape[1], D, A.shape[1], B.shape[-2],
                            1 if dt_softplus else 0)


def _scan_inputs(d, u, dt, A, B, C, D, z, dt_bias, step=False):
    """The leading arguments of the scan's calls, checked."""
    lead = (d.batch,) if step else (d.batch, d.seqlen)
    nd, view = d.channels, _token if step else _seq
    row, grp, io = (*lead, nd), (*lead, d.ngroups, d.dstate), u.dtype
    return [d, _io(u, "u"), view(u, "u", row, io, u), view(dt, "dt", row, io, u),
            _dense(A, "A", (nd, d.dstate), torch.float32, u), _grouped(B, "B", grp, io, u),
            _grouped(C, "C", grp, io, u), _dense(D, "D", (nd,), torch.float32, u),
            view(z, "z", row, io, u), _dense(dt_bias, "dt_bias", (nd,), torch.float32, u)]


def selective_scan_workspace_size(u, A, B) -> int:
    """Bytes of workspace that selective_scan_forward needs (may be 0)."""
    d = _scan_dims(u, A, B, False)
    return int(_abi.load().ssd_selective_scan_workspace_size(d, _io(u, "u")))


def selective_scan_forward(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None,
                           dt_softplus: bool = False, y=None, final_state=None,
                           return_final_state: bool = True, workspace=None):
    """y [b, L, D], final_state [b, D, N] = the scan whose decay is
    exp(s A[d, n]) per channel and state, with the step s = dt + dt_bias or
    softplus of it (ssd_selective_scan).

    u, dt, z [b, L, D] and B, C [b, L, G, N] in the I/O type (G groups of
    channels share B and C, N <= 64); A [D, N], D [D], dt_bias [D] and h0
    [b, D, N] float32.  With z, y is multiplied by silu(z).  final_state must
    not be h0."""
    d = _scan_dims(u, A, B, dt_softplus)
    _separate(final_state, "final_state", h0, "h0")
    lib, b, L, nd = _abi.load(), d.batch, d.seqlen, d.channels
    args = _scan_inputs(d, u, dt, A, B, C, D, z, dt_bias)
    keep = (b, nd, d.dstate)
    y = _out(y, "y", (b, L, nd), u.dtype, u)
    if final_state is None and return_final_state:
        final_state = torch.empty(keep, dtype=torch.float32, device=u.device)
    ws, wp, wn = _workspace(lib.ssd_selective_scan_workspace_size(d, args[1]), workspace, u,
                            "selective_scan_forward")
    _abi.check("ssd_selective_scan", lib.ssd_selective_scan(
        *args, _dense(h0, "h0", keep, torch.float32, u), _lengths(lengths, b, u),
        _seq(y, "y", (b, L, nd), u.dtype, u),
        _dense(final_state, "final_state", keep, torch.float32, u), wp, wn, _stream(u)))
    return y, final_state


_SCAN_GRADS = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


def selective_scan_backward_workspace_size(u, A, B) -> int:
    """Bytes of workspace that selective_scan_backward needs."""
    d = _scan_dims(u, A, B, False)
    return int(_abi.load().ssd_selective_scan_backward_workspace_size(d, _io(u, "u")))


def selective_scan_backward(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, gy=None,
                            gfinal=None, lengths=None, dt_softplus: bool = False,
                            workspace=None, want=None) -> dict:
    """Gradients through selective_scan_forward given gy = dL/dy and gfinal =
    dL/dfinal_state (None = 0), by ssd_selective_scan_backward: a dict of du,
    ddt, dB, dC, dz (I/O type), dA, dD, ddt_bias, dh0 (float32); those of
    absent inputs are None.  `want` names those to compute (None = all) and the
    others are None, but du, ddt, dB and dC are always computed."""
    if gy is None:
        raise ValueError("gy (dL/dy) is required")
    has = _wanted(want, _SCAN_GRADS, "selective_scan_backward")
    d = _scan_dims(u, A, B, dt_softplus)
    lib, b, L, nd, N = _abi.load(), d.batch, d.seqlen, d.channels, d.dstate
    args = _scan_inputs(d, u, dt, A, B, C, D, z, dt_bias)
    row, grp, keep = (b, L, nd), (b, L, d.ngroups, N), (b, nd, N)

    def io_out(shape, there=True):
        return torch.empty(shape, dtype=u.dtype, device=u.device) if there else None

    def f32_out(name, shape, of):
        return torch.empty(shape, dtype=torch.float32, device=u.device) \
            if has(name, of is not None) else None

    r = {"du": io_out(row), "ddt": io_out(row), "dA": f32_out("dA", (nd, N), A),
         "dB": io_out(grp), "dC": io_out(grp), "dD": f32_out("dD", (nd,), D),
         "dz": io_out(row, has("dz", z is not None)),
         "ddt_bias": f32_out("ddt_bias", (nd,), dt_bias), "dh0": f32_out("dh0", keep, h0)}
    g = _abi.SsdScanGrads()
    for k in ("du", "ddt", "dz"):
        if r[k] is not None:
            setattr(g, k, _seq(r[k], k, row, u.dtype, u))
    for k in ("dB", "dC"):
        setattr(g, k, _grouped(r[k], k, grp, u.dtype, u))
    for k in ("dA", "dD", "ddt_bias", "dh0"):
        if r[k] is not None:
            setattr(g, k, r[k].data_ptr())
    ws, wp, wn = _workspace(lib.ssd_selective_scan_backward_workspace_size(d, args[1]), workspace,
                            u, "selective_scan_backward")
    _abi.check("ssd_selective_scan_backward", lib.ssd_selective_scan_backward(
        *args, _dense(h0, "h0", keep, torch.float32, u), _seq(gy, "gy", row, u.dtype, u),
        _dense(gfinal, "gfinal", keep, torch.float32, u), _lengths(lengths, b, u), g, wp, wn,
        _stream(u)))
    return r


def selective_scan_step(u, dt, A, B, C, D, z, dt_bias, state, dt_softplus: bool = False, y=None):
    """y [b, D] = one token of the scan for every sequence
    (ssd_selective_scan_step).  u, dt, z [b, D], B, C [b, G, N]; state
    [b, D, N] float32 is updated in place.  D, z and dt_bias may be None."""
    if state is None:
        raise ValueError("state is required")
    d = _scan_dims(u, A, B, dt_softplus, step=True)
    args = _scan_inputs(d, u, dt, A, B, C, D, z, dt_bias, step=True)
    row = (d.batch, d.channels)
    y = _out(y, "y", row, u.dtype, u)
    _abi.check("ssd_selective_scan_step", _abi.load().ssd_selective_scan_step(
        *args, _dense(state, "state", (d.batch, d.channels, d.dstate), torch.float32, u),
        _token(y, "y", row, u.dtype, u), _stream(u)))
    return y


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, z, dt_bias, h0, lengths, dt_softplus):
        y, final_state = selective_scan_forward(u, dt, A, B, C, D, z, dt_bias, h0, lengths,
                                                dt_softplus)
        ctx.save_for_backward(u, dt, A, B, C, D, z, dt_bias, h0, lengths)
        ctx.dt_softplus = dt_softplus
        return y, final_state

    @staticmethod
    @_first_order
    def backward(ctx, gy, gfinal):
        *tensors, lengths = ctx.saved_tensors
        want = _needed(ctx, _SCAN_GRADS)
        g = selective_scan_backward(*tensors, gy.contiguous(), gfinal.contiguous(), lengths,
                                    ctx.dt_softplus, want=want)
        return (*(g[k] if k in want else None for k in _SCAN_GRADS), None, None)


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None,
                   dt_softplus: bool = False):
    """y, final_state = selective_scan_forward, differentiable with respect to
    u, dt, A, B, C, D, z, dt_bias and h0."""
    return _SelectiveScan.apply(u, dt, A, B, C, D, z, dt_bias, h0, lengths, dt_softplus)


# -------------------------------------------------------- gated group norm

def _norm_dims(x, groups, eps, gate, center):
    if gate not in _GATES:
        raise ValueError(f"gate must be 'none', 'input' or 'output', got {gate!r}")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [tokens, D] or [b, L, D]")
    b, L = (x.shape[0], 1) if x.dim() == 2 else x.shape[:2]
    return _abi.SsdNormDims(b, L, x.shape[-1], groups, eps, _GATES[gate], 1 if center else 0)


def _rows(d):
    """[tokens, D] runs as one sequence of that many tokens."""
    if d.seqlen == 1:
        d.batch, d.seqlen = 1, d.batch
        return True
    return False


def _check_gate(z, gate):
    if z is None and gate != "none":
        raise ValueError(f"gate {gate!r} needs z (without a gate: gate='none')")
    if z is not None and gate == "none":
        raise ValueError("z is given but gate is 'none'")


def _norm_view(t, name, x, flat):
    if x.dim() == 3:
        v = _seq(t, name, x.shape, x.dtype, x)
    else:
        v = _token(t, name, x.shape, x.dtype, x)
    if flat and v is not None:
        v.batch_stride, v.token_stride = 0, v.batch_stride
    return v


def gated_norm_forward(x, weight, bias=None, z=None, groups: int = 1, eps: float = 1e-5,
                       gate: str = "input", center: bool = False, y=None):
    """y = the group norm of every token over each of `groups` groups of
    channels, with a SiLU gate (ssd_gated_norm): gate "input" normalises
    x silu(z), "output" multiplies the result by silu(z), "none" takes no z.
    Root mean square, or centred with `center`.

    x, z [tokens, D] or [b, L, D] in the I/O type, weight and bias [D]
    float32.  y may be x or z themselves."""
    d = _norm_dims(x, groups, eps, gate, center)
    _check_gate(z, gate)
    flat, D = _rows(d), x.shape[-1]
    y = _out(y, "y", x.shape, x.dtype, x)
    _abi.check("ssd_gated_norm", _abi.load().ssd_gated_norm(
        d, _io(x, "x"), _norm_view(x, "x", x, flat),
        _dense(weight, "weight", (D,), torch.float32, x),
        _dense(bias, "bias", (D,), torch.float32, x), _norm_view(z, "z", x, flat),
        _norm_view(y, "y", x, flat), _stream(x)))
    return y


_NORM_GRADS = ("dx", "dweight", "dbias", "dz")


def gated_norm_backward_workspace_size(x, groups: int = 1) -> int:
    """Bytes of workspace that gated_norm_backward needs."""
    d = _norm_dims(x, groups, 1e-5, "none", False)
    _rows(d)
    return int(_abi.load().ssd_gated_norm_backward_workspace_size(d, _io(x, "x")))


def gated_norm_backward(x, weight, bias=None, z=None, gy=None, groups: int = 1,
                        eps: float = 1e-5, gate: str = "input", center: bool = False,
                        workspace=None, want=None) -> dict:
    """Gradients through gated_norm_forward given gy = dL/dy, by
    ssd_gated_norm_backward: a dict of dx, dz (I/O type; dz None without a
    gate), dweight and dbias (float32; dbias None without a bias).  `want` names
    those to compute (None = all) and the others are None, but dx and dz are
    always computed."""
    if gy is None:
        raise ValueError("gy (dL/dy) is required")
    has = _wanted(want, _NORM_GRADS, "gated_norm_backward")
    d = _norm_dims(x, groups, eps, gate, center)
    _check_gate(z, gate)
    flat, D, lib, io = _rows(d), x.shape[-1], _abi.load(), _io(x, "x")
    ws, wp, wn = _workspace(lib.ssd_gated_norm_backward_workspace_size(d, io), workspace, x,
                            "gated_norm_backward")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dz = None if z is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw, db = (torch.empty((D,), dtype=torch.float32, device=x.device) if has(name, there) else None
              for name, there in (("dweight", True), ("dbias", bias is not None)))
    _abi.check("ssd_gated_norm_backward", lib.ssd_gated_norm_backward(
        d, io, _norm_view(x, "x", x, flat), _dense(weight, "weight", (D,), torch.float32, x),
        _dense(bias, "bias", (D,), torch.float32, x), _norm_view(z, "z", x, flat),
        _norm_view(gy, "gy", x, flat), _norm_view(dx, "dx", x, flat),
        _norm_view(dz, "dz", x, flat), *(None if t is None else t.data_ptr() for t in (dw, db)),
        wp, wn, _stream(x)))
    return {"dx": dx, "dz": dz, "dweight": dw, "dbias": db}


class _GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, z, groups, eps, gate, center):
        ctx.save_for_backward(x, weight, bias, z)
        ctx.how = (groups, eps, gate, center)
        return gated_norm_forward(x, weight, bias, z, *ctx.how)

    @staticmethod
    @_first_order
    def backward(ctx, gy):
        x, weight, bias, z = ctx.saved_tensors
        want = _needed(ctx, _NORM_GRADS)
        g = gated_norm_backward(x, weight, bias, z, gy.contiguous(), *ctx.how, want=want)
        return (*(g[k] if k in want else None for k in _NORM_GRADS), None, None, None, None)


def gated_norm(x, weight, bias=None, z=None, groups: int = 1, eps: float = 1e-5,
               gate: str = "input", center: bool = False):
    """gated_norm_forward, differentiable with respect to x, weight, bias and
    z."""
    return _GatedNorm.apply(x, weight, bias, z, groups, eps, gate, center)


# ------------------------------------------- gradient norm and clipping

def clip_grad_norm_workspace_size(grads) -> int:
    """Bytes of workspace that clip_grad_norm needs for tensors of these sizes
    and types."""
    table = (_abi.SsdGrad * len(grads))(*((256, 256, g.numel(), _io(g, "grads"))
                                          for g in grads))  # any aligned address will do
    return int(_abi.load().ssd_clip_grad_norm_workspace_size(table, len(grads)))


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, out=None, workspace=None):
    """The norm over every element of every tensor of `grads` (a float32
    scalar on the device), and the tensors scaled by min(1, max_norm / (norm +
    eps)) (ssd_clip_grad_norm): in place, or into the tensors of `out`.

    Contiguous float32 or bfloat16 tensors of any shapes, mixed; empty ones
    are skipped.  A tensor may be given once only.  Nothing waits for the
    device."""
    grads = list(grads)
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError(f"{len(grads)} gradients but {len(out)} outputs")
    if not grads:
        raise ValueError("no gradients given")
    like = grads[0]
    dev, flat = like.get_device(), []
    if dev < 0:
        _io(like, "grads[0]")
        _refuse(like, "grads[0]", like.shape, like.dtype, like)
    for g, o in zip(grads, out):
        io = _IO.get(g.dtype)
        if io is None or g.get_device() != dev or not g.is_contiguous():
            i = next(i for i, t in enumerate(grads) if t is g)
            _io(g, f"grads[{i}]")
            _refuse(g, f"grads[{i}]", g.shape, g.dtype, like)
        src = dst = g.data_ptr()
        if o is not g:
            if (o.dtype is not g.dtype or o.get_device() != dev or not o.is_contiguous()
                    or o.shape != g.shape):
                i = next(i for i, t in enumerate(out) if t is o)
                _refuse(o, f"out[{i}]", g.shape, g.dtype, like)
            dst = o.data_ptr()
        flat += (src, dst, g.numel(), io)
    n = len(grads)
    if len(set(flat[1::4])) < n:  # empty tensors may share an address
        written = [at for at, k in zip(flat[1::4], flat[2::4]) if k]
        if len(set(written)) < len(written):
            raise ValueError("a tensor is given more than once: it would be scaled twice at once")
    table = (_abi.SsdGrad * n).from_buffer_copy(struct.pack("@" + "PPqi4x" * n, *flat))
    lib = _abi.load()
    norm = torch.empty((), dtype=torch.float32, device=like.device)
    ws, wp, wn = _workspace(lib.ssd_clip_grad_norm_workspace_size(table, n), workspace,
                            like, "clip_grad_norm")
    _abi.check("ssd_clip_grad_norm", lib.ssd_clip_grad_norm(
        table, n, max_norm, eps, norm.data_ptr(), wp, wn, _stream(like)))
    return norm
