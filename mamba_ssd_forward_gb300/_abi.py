"""ctypes view of the C ABI declared in include/ssd.h and include/ssd_layer.h
(libssd_gb300.so).

Marshalling only: every step of the forward pass runs in the library's CUDA
kernels.  If the library has not been built, loading fails loudly; there is
no fallback.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libssd_gb300.so")

(SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_CUDA, SSD_ERR_TIMEOUT,
 SSD_ERR_BOUNDS) = range(6)
SSD_F32, SSD_BF16 = 0, 1
# Size of the fixed scratch array of ssd_forward_noalloc (SSD_NOALLOC_SCRATCH_BYTES).
SSD_NOALLOC_SCRATCH_BYTES = 32 << 20
# Workspace header holding a call's device error word (SSD_WS_HEADER_BYTES).
SSD_WS_HEADER_BYTES = 256

# Every symbol include/ssd.h and include/ssd_layer.h declare.
EXPORTS = (
    "ssd_status_string",
    "ssd_forward_workspace_size",
    "ssd_chunk_cumsum",
    "ssd_chunk_state",
    "ssd_state_passing",
    "ssd_chunk_scan",
    "ssd_forward",
    "ssd_forward_ex",
    "ssd_workspace_error",
    "ssd_device_error",
    "ssd_forward_profiled",
    "ssd_forward_host_workspace_size",
    "ssd_forward_host",
    "ssd_forward_noalloc",
    "ssd_decode_step",
    "ssd_forward_host_overlapped_workspace_size",
    "ssd_forward_host_overlapped",
    "ssd_forward_plan_candidates",
    "ssd_forward_default_plan",
    "ssd_forward_tune",
    "ssd_selftest_bounded_wait",
    "ssd_backward_workspace_size",
    "ssd_backward",
    "ssd_backward_profiled",
    "ssd_causal_conv",
    "ssd_causal_conv_backward_workspace_size",
    "ssd_causal_conv_backward",
    "ssd_causal_conv_step",
    "ssd_selective_scan_workspace_size",
    "ssd_selective_scan",
    "ssd_selective_scan_backward_workspace_size",
    "ssd_selective_scan_backward",
    "ssd_selective_scan_step",
    "ssd_gated_norm",
    "ssd_gated_norm_backward_workspace_size",
    "ssd_gated_norm_backward",
    "ssd_clip_grad_norm_workspace_size",
    "ssd_clip_grad_norm",
    "ssd_add_norm",
    "ssd_add_norm_quantized",
    "ssd_add_norm_backward_workspace_size",
    "ssd_add_norm_backward",
    "ssd_linear_cross_entropy_workspace_size",
    "ssd_linear_cross_entropy",
    "ssd_linear_cross_entropy_backward_workspace_size",
    "ssd_linear_cross_entropy_backward",
    "ssd_orthogonalize_workspace_size",
    "ssd_orthogonalize",
)

SSD_ACT_NONE, SSD_ACT_SILU = 0, 1
SSD_GATE_NONE, SSD_GATE_INPUT, SSD_GATE_OUTPUT = 0, 1, 2
SSD_REDUCE_NONE, SSD_REDUCE_SUM, SSD_REDUCE_MEAN = 0, 1, 2


class SsdDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "seqlen", "nheads", "headdim", "dstate", "ngroups", "chunk")]


class SsdPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("chunk_state_heads", "chunk_state_ctas", "scan_kernel", "scan_heads")]

    def as_dict(self) -> dict:
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


class SsdSeq(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class SsdConvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "channels", "width")] + \
        [("activation", ctypes.c_int32)]


class SsdScanDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "seqlen", "channels", "dstate", "ngroups")] + \
        [("dt_softplus", ctypes.c_int32)]


class SsdScanGrads(ctypes.Structure):
    _fields_ = [(n, SsdSeq) for n in ("du", "ddt", "dz", "dB", "dC")] + \
        [(n, ctypes.c_void_p) for n in ("dA", "dD", "ddt_bias", "dh0")]


class SsdNormDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "channels", "ngroups")] + \
        [("eps", ctypes.c_float), ("gate", ctypes.c_int32), ("center", ctypes.c_int32)]


class SsdGrad(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class SsdAddNormDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "channels")] + \
        [("eps", ctypes.c_float)]


class SsdLossDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "seqlen", "channels", "vocab", "ignore_index")] + \
        [("reduction", ctypes.c_int32)]


class SsdOrthDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("count", "rows", "cols")] + \
        [("steps", ctypes.c_int32)] + [(n, ctypes.c_float) for n in ("a", "b", "c", "eps")]


class SsdError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


_lib = None


def load(path: str | None = None):
    """Load libssd_gb300.so and declare its prototypes."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build the CUDA library first "
            "(python -m mamba_ssd_forward_gb300.build, or __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    vp, dims_p, i32, sz = ctypes.c_void_p, ctypes.POINTER(SsdDims), ctypes.c_int, ctypes.c_size_t
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [i32]
    lib.ssd_forward_workspace_size.restype = sz
    lib.ssd_forward_workspace_size.argtypes = [dims_p, i32]
    lib.ssd_chunk_cumsum.restype = i32
    lib.ssd_chunk_cumsum.argtypes = [dims_p, i32, vp, vp, vp, vp]
    lib.ssd_chunk_state.restype = i32
    lib.ssd_chunk_state.argtypes = [dims_p, i32, vp, vp, vp, vp, vp, vp]
    lib.ssd_state_passing.restype = i32
    lib.ssd_state_passing.argtypes = [dims_p, vp, vp, vp, vp, vp, vp]
    lib.ssd_chunk_scan.restype = i32
    lib.ssd_chunk_scan.argtypes = [dims_p, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    plan_p = ctypes.POINTER(SsdPlan)
    lib.ssd_forward.restype = i32
    lib.ssd_forward.argtypes = [dims_p, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ssd_forward_ex.restype = i32
    lib.ssd_forward_ex.argtypes = [dims_p, i32] + [vp] * 10 + [sz, plan_p, vp]
    lib.ssd_workspace_error.restype = i32
    lib.ssd_workspace_error.argtypes = [vp, vp]
    lib.ssd_device_error.restype = i32
    lib.ssd_device_error.argtypes = [vp]
    lib.ssd_forward_profiled.restype = i32
    lib.ssd_forward_profiled.argtypes = ([dims_p, i32] + [vp] * 10 + [sz, plan_p, vp, vp, i32,
                                         ctypes.POINTER(ctypes.c_int)])
    lib.ssd_forward_host_workspace_size.restype = sz
    lib.ssd_forward_host_workspace_size.argtypes = [dims_p, i32, i32, i32, i32]
    lib.ssd_forward_host.restype = i32
    lib.ssd_forward_host.argtypes = [dims_p, i32] + [vp] * 10 + [sz, plan_p, vp]
    lib.ssd_forward_host_overlapped_workspace_size.restype = sz
    lib.ssd_forward_host_overlapped_workspace_size.argtypes = [dims_p, i32, i32, i32, i32, i32]
    lib.ssd_forward_host_overlapped.restype = i32
    lib.ssd_forward_host_overlapped.argtypes = ([dims_p, i32] + [vp] * 10 +
                                                [sz, i32, plan_p, vp, vp, vp])
    lib.ssd_decode_step.restype = i32
    lib.ssd_decode_step.argtypes = [dims_p, i32] + [vp] * 9
    lib.ssd_forward_noalloc.restype = i32
    lib.ssd_forward_noalloc.argtypes = [dims_p, i32] + [vp] * 9 + [vp]
    lib.ssd_forward_plan_candidates.restype = i32
    lib.ssd_forward_plan_candidates.argtypes = [dims_p, i32, plan_p, i32]
    lib.ssd_forward_default_plan.restype = i32
    lib.ssd_forward_default_plan.argtypes = [dims_p, i32, plan_p]
    lib.ssd_selftest_bounded_wait.restype = i32
    lib.ssd_selftest_bounded_wait.argtypes = [ctypes.c_uint64, vp, vp]
    lib.ssd_forward_tune.restype = i32
    lib.ssd_forward_tune.argtypes = [dims_p, i32] + [vp] * 10 + [sz, i32, vp, sz, vp, plan_p]
    lib.ssd_backward_workspace_size.restype = sz
    lib.ssd_backward_workspace_size.argtypes = [dims_p, i32]
    lib.ssd_backward.restype = i32
    lib.ssd_backward.argtypes = [dims_p, i32] + [vp] * 17 + [sz, vp]
    lib.ssd_backward_profiled.restype = i32
    lib.ssd_backward_profiled.argtypes = ([dims_p, i32] + [vp] * 17 +
                                          [sz, vp, vp, i32, ctypes.POINTER(ctypes.c_int)])
    P = ctypes.POINTER
    seq, conv, scan, norm = P(SsdSeq), P(SsdConvDims), P(SsdScanDims), P(SsdNormDims)
    f32, i64 = ctypes.c_float, ctypes.c_int64
    add, loss, orth = P(SsdAddNormDims), P(SsdLossDims), P(SsdOrthDims)
    for name, res, args in (
            ("ssd_causal_conv", i32, [conv, i32, seq, vp, vp, vp, vp, seq, vp, vp]),
            ("ssd_causal_conv_backward_workspace_size", sz, [conv, i32]),
            ("ssd_causal_conv_backward", i32,
             [conv, i32, seq, vp, vp, vp, seq, vp, vp, seq, vp, vp, vp, vp, sz, vp]),
            ("ssd_causal_conv_step", i32, [conv, i32, seq, vp, vp, vp, seq, vp]),
            ("ssd_selective_scan_workspace_size", sz, [scan, i32]),
            ("ssd_selective_scan", i32,
             [scan, i32, seq, seq, vp, seq, seq, vp, seq, vp, vp, vp, seq, vp, vp, sz, vp]),
            ("ssd_selective_scan_backward_workspace_size", sz, [scan, i32]),
            ("ssd_selective_scan_backward", i32,
             [scan, i32, seq, seq, vp, seq, seq, vp, seq, vp, vp, seq, vp, vp, P(SsdScanGrads),
              vp, sz, vp]),
            ("ssd_selective_scan_step", i32,
             [scan, i32, seq, seq, vp, seq, seq, vp, seq, vp, vp, seq, vp]),
            ("ssd_gated_norm", i32, [norm, i32, seq, vp, vp, seq, seq, vp]),
            ("ssd_gated_norm_backward_workspace_size", sz, [norm, i32]),
            ("ssd_gated_norm_backward", i32,
             [norm, i32, seq, vp, vp, seq, seq, seq, seq, vp, vp, vp, sz, vp]),
            ("ssd_clip_grad_norm_workspace_size", sz, [P(SsdGrad), i32]),
            ("ssd_clip_grad_norm", i32, [P(SsdGrad), i32, f32, f32, vp, vp, sz, vp]),
            ("ssd_add_norm", i32, [add, i32, i32, seq, seq, vp, seq, seq, vp]),
            ("ssd_add_norm_quantized", i32,
             [add, i32, i32, i64, seq, seq, vp, seq, vp, seq, vp]),
            ("ssd_add_norm_backward_workspace_size", sz, [add, i32, i32]),
            ("ssd_add_norm_backward", i32,
             [add, i32, i32, seq, vp, seq, seq, seq, seq, vp, vp, sz, vp]),
            ("ssd_linear_cross_entropy_workspace_size", sz, [loss, i32, seq]),
            ("ssd_linear_cross_entropy", i32,
             [loss, i32, seq, seq, vp, vp, vp, vp, vp, sz, vp]),
            ("ssd_linear_cross_entropy_backward_workspace_size", sz, [loss, i32, seq]),
            ("ssd_linear_cross_entropy_backward", i32,
             [loss, i32, seq, seq, vp, vp, vp, seq, vp, vp, sz, vp]),
            ("ssd_orthogonalize_workspace_size", sz, [orth, i32, i32]),
            ("ssd_orthogonalize", i32, [orth, i32, i32, seq, seq, vp, sz, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    if path is None:
        _lib = lib
    return lib


def check(fn: str, code: int) -> None:
    if code != SSD_OK:
        msg = load().ssd_status_string(code).decode()
        raise SsdError(fn, code, msg)
