"""The operators around the blocks of a language model (include/ssd_model.h):
the residual's addition with the norm in front of a block, the cross entropy
over a large vocabulary without its logits, and the orthogonalisation of an
update.

As in layer.py, the functions check types and shapes, allocate outputs and
workspaces on the current CUDA stream and pass pointers; all arithmetic runs
in the library's kernels.  Activations are [tokens, D] or [b, L, D] views with
any strides between sequences and tokens as long as the last axis is dense.
"""
from __future__ import annotations

import torch

from . import _abi
from ._abi import SsdAddNormDims, SsdSeq
from .layer import (_IO, _dense, _first_order, _io, _needed, _out, _refuse, _seq, _separate,
                    _stream, _token, _wanted, _workspace)

_REDUCTIONS = {"none": _abi.SSD_REDUCE_NONE, "sum": _abi.SSD_REDUCE_SUM,
               "mean": _abi.SSD_REDUCE_MEAN}


def _lead(x, name):
    """Sequences and tokens of [tokens, D] (one sequence) or [b, L, D]."""
    if x.dim() not in (2, 3):
        raise ValueError(f"{name} must be [tokens, D] or [b, L, D]")
    b, L, D = x.shape if x.dim() == 3 else (1, *x.shape)
    if not b * L * D:
        raise ValueError(f"{name} must not be empty")
    return b, L


def _view(t, name, shape, dtype, like):
    """View of an activation; [tokens, D] as one sequence.  None stays None."""
    if t is None:
        return None
    if len(shape) == 3:
        return _seq(t, name, shape, dtype, like)
    v = _token(t, name, shape, dtype, like)
    v.batch_stride, v.token_stride = 0, v.batch_stride
    return v


# -------------------------------------------------- residual addition and norm

# A call for a few tokens takes 5 us on the device, so these keep to as few Python
# steps as their checks allow.

def _stream_type(x, stream):
    """The residual stream's type: that of x, or float32."""
    if stream is not x.dtype and stream is not torch.float32:
        raise TypeError(f"the residual must be {x.dtype} or torch.float32, got {stream}")
    return stream


def _add_norm_dims(x, eps):
    b, L = _lead(x, "x")
    return SsdAddNormDims(b, L, x.shape[-1], eps)


def _rows(t, name, shape, dtype, dev, like):
    """View of [tokens, D] or [b, L, D]; what else it may be is refused."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or dev < 0:
        _refuse(t, name, shape, dtype, like)
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        _refuse(t, name, shape, dtype, like)
    if len(st) == 2:
        return SsdSeq(t.data_ptr(), 0, st[0] if shape[0] > 1 else 0)
    return SsdSeq(t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0)


def _in_place(out, name, source, source_name):
    """Refuses an output at the address of an input that it may be, unless it is
    that view: rows elsewhere are other threads' to read."""
    if (source is not None and out.data_ptr() == source.data_ptr()
            and any(a != b for a, b, n in zip(out.stride(), source.stride(), out.shape) if n > 1)):
        raise ValueError(f"{name} must be {source_name} itself or other memory")


def _new_rows(shape, dtype, like):
    """A new dense tensor of that shape, and its view."""
    t = torch.empty(shape, dtype=dtype, device=like.device)
    D = shape[-1]
    return t, SsdSeq(t.data_ptr(), shape[1] * D if len(shape) == 3 else 0, D)


def _add_norm_inputs(x, residual, weight, total, eps):
    """What both forward calls check and pass, total, and what they share."""
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    d, io = _add_norm_dims(x, eps), _io(x, "x")
    like = residual if residual is not None else total
    stream = dtype if like is None else _stream_type(x, like.dtype)
    xv = _rows(x, "x", shape, dtype, dev, x)
    rv = None if residual is None else _rows(residual, "residual", shape, stream, dev, x)
    if (weight.dtype is not torch.float32 or weight.dim() != 1 or len(weight) != shape[-1]
            or weight.stride(0) != 1 or weight.get_device() != dev):
        _dense(weight, "weight", shape[-1:], torch.float32, x)
    tv = None
    if total is not None:
        _out(total, "total", shape, stream, x)
        _separate(total, "total", x, "x")
        _in_place(total, "total", residual, "residual")
        tv = _rows(total, "total", shape, stream, dev, x)
    elif residual is not None:
        total, tv = _new_rows(shape, stream, x)
    return (d, io, _IO[stream]), (xv, rv, weight.data_ptr()), total, tv, shape, dev


def add_norm_forward(x, residual, weight, eps: float = 1e-5, y=None, total=None):
    """y = the root-mean-square norm of x + residual, times weight, and total =
    x + residual, the residual of the next block (ssd_add_norm).

    x [tokens, D] or [b, L, D] in the I/O type; residual and total of the same
    shape, in the I/O type or float32; weight [D] float32.  The norm is that of the
    sum before total's rounding.  Without a residual (None) total is None
    unless it is given.  y may be x, total may be residual."""
    head, ins, total, tv, shape, dev = _add_norm_inputs(x, residual, weight, total, eps)
    if y is None:
        y, yv = _new_rows(shape, x.dtype, x)
    else:
        _out(y, "y", shape, x.dtype, x)
        _separate(y, "y", residual, "residual")
        _separate(y, "y", total, "total")
        _in_place(y, "y", x, "x")
        yv = _rows(y, "y", shape, x.dtype, dev, x)
    code = _abi.load().ssd_add_norm(*head, *ins, yv, tv, _stream(x))
    if code:
        _abi.check("ssd_add_norm", code)
    return y, total


def add_norm_quantized(x, residual, weight, block: int = 128, eps: float = 1e-5, q=None,
                       scales=None, total=None):
    """add_norm_forward with y in 8 bits (ssd_add_norm_quantized): q
    (float8_e4m3fn, the shape of x), scales (float32 [.., ceil(D / block)]) and
    total.  y is q times its block's scale, which is max|y| / 448 over `block`
    channels (32, 64 or 128) or, with block = 0, over the token.  q and scales
    have memory of their own."""
    if block not in (0, 32, 64, 128):
        raise ValueError(f"block must be 0, 32, 64 or 128, got {block!r}")
    head, ins, total, tv, shape, dev = _add_norm_inputs(x, residual, weight, total, eps)
    *lead, D = shape
    lead.append(-(-D // block) if block else 1)
    if scales is None:
        scales = torch.empty(lead, dtype=torch.float32, device=x.device)
        at = scales.data_ptr()
    else:
        at = _dense(scales, "scales", tuple(lead), torch.float32, x)
        for t, name in ((x, "x"), (residual, "residual"), (total, "total")):
            _separate(scales, "scales", t, name)
    if q is None:
        q, qv = _new_rows(shape, torch.float8_e4m3fn, x)
    else:
        _out(q, "q", shape, torch.float8_e4m3fn, x)
        for t, name in ((x, "x"), (residual, "residual"), (total, "total"), (scales, "scales")):
            _separate(q, "q", t, name)
        qv = _rows(q, "q", shape, torch.float8_e4m3fn, dev, x)
    code = _abi.load().ssd_add_norm_quantized(*head, block, *ins, qv, at, tv, _stream(x))
    if code:
        _abi.check("ssd_add_norm_quantized", code)
    return q, scales, total


_ADD_NORM_GRADS = ("dx", "dresidual", "dweight")


def add_norm_backward_workspace_size(total, gy) -> int:
    """Bytes of workspace that add_norm_backward needs."""
    return int(_abi.load().ssd_add_norm_backward_workspace_size(
        _add_norm_dims(gy, 1e-5), _io(gy, "gy"), _IO[_stream_type(gy, total.dtype)]))


def add_norm_backward(total, weight, gy, gtotal=None, eps: float = 1e-5, workspace=None,
                      want=None) -> dict:
    """Gradients through add_norm_forward from its total, given gy = dL/dy (the
    I/O type) and gtotal = dL/dtotal (total's type; None = 0), by
    ssd_add_norm_backward: a dict of dx (the I/O type), dresidual (total's
    type; where the types are the same, the same tensor) and dweight
    (float32).  `want` names those to compute (None = all)."""
    has = _wanted(want, _ADD_NORM_GRADS, "add_norm_backward")
    d, io, lib = _add_norm_dims(gy, eps), _io(gy, "gy"), _abi.load()
    stream, shape, dtype, dev = _stream_type(gy, total.dtype), gy.shape, gy.dtype, gy.get_device()
    st, one = _IO[stream], stream is dtype
    ins = (_rows(total, "total", shape, stream, dev, gy),
           _dense(weight, "weight", shape[-1:], torch.float32, gy),
           _rows(gy, "gy", shape, dtype, dev, gy),
           None if gtotal is None else _rows(gtotal, "gtotal", shape, stream, dev, gy))
    dx = xv = dr = rv = dw = ws = None
    wp, wn = None, 0
    if has("dx") or (one and has("dresidual")):
        dx, xv = _new_rows(shape, dtype, gy)
    if has("dresidual") and not one:
        dr, rv = _new_rows(shape, stream, gy)
    if has("dweight"):
        dw = torch.empty(shape[-1:], dtype=torch.float32, device=gy.device)
        ws, wp, wn = _workspace(lib.ssd_add_norm_backward_workspace_size(d, io, st), workspace,
                                gy, "add_norm_backward")
    code = lib.ssd_add_norm_backward(d, io, st, *ins, xv, rv,
                                     None if dw is None else dw.data_ptr(), wp, wn, _stream(gy))
    if code:
        _abi.check("ssd_add_norm_backward", code)
    dr = dx if one else dr
    return {"dx": dx if has("dx") else None, "dresidual": dr if has("dresidual") else None,
            "dweight": dw}


class _AddNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, total = add_norm_forward(x, residual, weight, eps)
        ctx.save_for_backward(total, weight)
        ctx.eps, ctx.io = eps, x.dtype
        ctx.set_materialize_grads(False)  # (behind the last block nothing uses total)
        return y, total

    @staticmethod
    @_first_order
    def backward(ctx, gy, gtotal):
        total, weight = ctx.saved_tensors
        gy = torch.zeros_like(total, dtype=ctx.io) if gy is None else gy.contiguous()
        gtotal = None if gtotal is None else gtotal.contiguous()
        g = add_norm_backward(total, weight, gy, gtotal, ctx.eps,
                              want=_needed(ctx, _ADD_NORM_GRADS))
        return (*(g[k] for k in _ADD_NORM_GRADS), None)


def add_norm(x, residual, weight, eps: float = 1e-5):
    """y, total = add_norm_forward, differentiable with respect to x, residual
    and weight.  residual is required (zeros in front of the first block)."""
    if residual is None:
        raise ValueError("residual is required (zeros in front of the first block)")
    return _AddNorm.apply(x, residual, weight, eps)


# ------------------------------------------------ cross entropy over a vocabulary

def _loss_dims(x, weight, ignore_index, reduction):
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be 'none', 'sum' or 'mean', got {reduction!r}")
    b, L = _lead(x, "x")
    if weight.dim() != 2 or not weight.shape[0]:
        raise ValueError("weight must be [V, D]")
    return _abi.SsdLossDims(b, L, x.shape[-1], weight.shape[0], ignore_index,
                            _REDUCTIONS[reduction])


def _words(weight, x):
    """View of the vocabulary's rows."""
    return _view(weight, "weight", (weight.shape[0], x.shape[-1]), x.dtype, x)


def linear_cross_entropy_workspace_size(x, weight) -> int:
    """Bytes of workspace that linear_cross_entropy_forward needs."""
    return int(_abi.load().ssd_linear_cross_entropy_workspace_size(
        _loss_dims(x, weight, -100, "none"), _io(x, "x"), _words(weight, x)))


def linear_cross_entropy_forward(x, weight, targets, ignore_index: int = -100,
                                 reduction: str = "none", workspace=None):
    """loss, lse = the softmax cross entropy of the logits x weight^T against
    targets, whose logits are not stored (ssd_linear_cross_entropy).

    x [tokens, D] or [b, L, D] and weight [V, D] in the I/O type, targets
    int64 of x's leading shape.  loss: float32 of that shape (reduction
    "none"), or its sum, or its mean over the tokens with a target ("mean"; 0
    without any).  lse: the logarithm of the sum of exponentials, float32, for
    the backward pass.  Tokens whose target is ignore_index have a loss and an
    lse of zero; another target outside [0, V) gives a NaN."""
    d, io, lib = _loss_dims(x, weight, ignore_index, reduction), _io(x, "x"), _abi.load()
    lead, w = x.shape[:-1], _words(weight, x)
    lse = torch.empty(lead, dtype=torch.float32, device=x.device)
    loss = torch.empty(lead if reduction == "none" else (), dtype=torch.float32, device=x.device)
    ws, wp, wn = _workspace(lib.ssd_linear_cross_entropy_workspace_size(d, io, w), workspace, x,
                            "linear_cross_entropy_forward")
    out = loss.data_ptr()
    _abi.check("ssd_linear_cross_entropy", lib.ssd_linear_cross_entropy(
        d, io, _view(x, "x", x.shape, x.dtype, x), w,
        _dense(targets, "targets", lead, torch.int64, x),
        *((out, None) if reduction == "none" else (None, out)), lse.data_ptr(), wp, wn,
        _stream(x)))
    return loss, lse


_LOSS_GRADS = ("dx", "dweight")


def linear_cross_entropy_backward_workspace_size(x, weight) -> int:
    """Bytes of workspace that linear_cross_entropy_backward needs."""
    return int(_abi.load().ssd_linear_cross_entropy_backward_workspace_size(
        _loss_dims(x, weight, -100, "none"), _io(x, "x"), _words(weight, x)))


def linear_cross_entropy_backward(x, weight, targets, lse, gloss=None, ignore_index: int = -100,
                                  reduction: str = "none", workspace=None, want=None) -> dict:
    """Gradients through linear_cross_entropy_forward from its lse, given gloss
    = dL/dloss (float32 of loss's shape; None = 1), by
    ssd_linear_cross_entropy_backward: a dict of dx (zero for tokens without a
    target) and dweight [V, D], both in the I/O type.  `want` names those to
    compute (None = both)."""
    has = _wanted(want, _LOSS_GRADS, "linear_cross_entropy_backward")
    d, io, lib = _loss_dims(x, weight, ignore_index, reduction), _io(x, "x"), _abi.load()
    lead, w = x.shape[:-1], _words(weight, x)
    ws, wp, wn = _workspace(lib.ssd_linear_cross_entropy_backward_workspace_size(d, io, w),
                            workspace, x, "linear_cross_entropy_backward")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if has("dx") else None
    dw = torch.empty(weight.shape, dtype=x.dtype, device=x.device) if has("dweight") else None
    _abi.check("ssd_linear_cross_entropy_backward", lib.ssd_linear_cross_entropy_backward(
        d, io, _view(x, "x", x.shape, x.dtype, x), w,
        _dense(targets, "targets", lead, torch.int64, x),
        _dense(lse, "lse", lead, torch.float32, x),
        _dense(gloss, "gloss", lead if reduction == "none" else (), torch.float32, x),
        _view(dx, "dx", x.shape, x.dtype, x), None if dw is None else dw.data_ptr(), wp, wn,
        _stream(x)))
    return {"dx": dx, "dweight": dw}


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, reduction):
        loss, lse = linear_cross_entropy_forward(x, weight, targets, ignore_index, reduction)
        ctx.save_for_backward(x, weight, targets, lse)
        ctx.how = (ignore_index, reduction)
        return loss

    @staticmethod
    @_first_order
    def backward(ctx, gloss):
        x, weight, targets, lse = ctx.saved_tensors
        g = linear_cross_entropy_backward(x, weight, targets, lse, gloss.contiguous(), *ctx.how,
                                          want=_needed(ctx, _LOSS_GRADS))
        return (*(g[k] for k in _LOSS_GRADS), None, None, None)


def linear_cross_entropy(x, weight, targets, ignore_index: int = -100, reduction: str = "mean"):
    """The loss of linear_cross_entropy_forward, differentiable with respect to
    x and weight."""
    return _LinearCrossEntropy.apply(x, weight, targets, ignore_index, reduction)


# ----------------------------------------------------- orthogonalised updates

#: The coefficients of a step, which take singular values near 1 fast.
ORTH_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _orth_dims(update, steps, coefficients, eps):
    if update.dim() not in (2, 3) or not update.numel():
        raise ValueError("update must be [rows, cols] or [k, rows, cols], not empty")
    k = 1 if update.dim() == 2 else update.shape[0]
    return _abi.SsdOrthDims(k, *update.shape[-2:], steps, *coefficients, eps)


def _result_type(update, dtype, out):
    dtype = dtype or (update.dtype if out is None else out.dtype)
    if dtype not in _IO:
        raise TypeError(f"the result must be float32 or bfloat16, got {dtype}")
    return dtype


def orthogonalize_workspace_size(update, dtype=None) -> int:
    """Bytes of workspace that orthogonalize needs."""
    dtype = _result_type(update, dtype, None)
    return int(_abi.load().ssd_orthogonalize_workspace_size(
        _orth_dims(update, 1, ORTH_COEFFICIENTS, 1e-7), _io(update, "update"), _IO[dtype]))


def orthogonalize(update, steps: int = 5, coefficients=ORTH_COEFFICIENTS, eps: float = 1e-7,
                  dtype=None, out=None, workspace=None):
    """The update with its singular values taken near 1 by Newton-Schulz steps
    (ssd_orthogonalize): X = G / (|G| + eps), then `steps` times X <- a X + b
    (X X^T) X + c (X X^T)^2 X, for a matrix [rows, cols] or each of a stack
    [k, rows, cols], float32 or bfloat16 with dense rows.

    The result is of `dtype` (None: that of out, or of update).  bfloat16 takes
    products of 11-bit operands, float32 of 22-bit ones at three times the work.
    out may be update where the types are the same."""
    d, io = _orth_dims(update, steps, coefficients, eps), _io(update, "update")
    dtype, lib, shape = _result_type(update, dtype, out), _abi.load(), update.shape
    out = _out(out, "out", shape, dtype, update)
    if out.dtype != update.dtype:
        _separate(out, "out", update, "update")
    ws, wp, wn = _workspace(lib.ssd_orthogonalize_workspace_size(d, io, _IO[dtype]), workspace,
                            update, "orthogonalize")
    _abi.check("ssd_orthogonalize", lib.ssd_orthogonalize(
        d, io, _IO[dtype], _view(update, "update", shape, update.dtype, update),
        _view(out, "out", shape, dtype, update), wp, wn, _stream(update)))
    return out
