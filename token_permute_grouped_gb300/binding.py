"""ctypes binding of liba2av_gmm.so: argument marshalling only.

Same names as the C ABI in include/*.h.  Every step of the hot path
runs in the library's CUDA kernels; this module only checks tensors, sizes the
outputs and workspace with torch, and passes raw device pointers and the
current CUDA stream.  There is no CPU fallback: without the built library
every entry point raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

from . import build as _build

A2AV_OK = 0
STATUS_NAMES = {0: "A2AV_OK", 1: "A2AV_ERR_NULLPTR", 2: "A2AV_ERR_INVALID", 3: "A2AV_ERR_UNSUPPORTED",
                4: "A2AV_ERR_WORKSPACE", 5: "A2AV_ERR_CUDA", 6: "A2AV_ERR_DEVICE_CHECK",
                7: "A2AV_ERR_SCRATCH_LIMIT", 8: "A2AV_ERR_ARRIVAL_TIMEOUT"}
STATIC_SCRATCH_BYTES = 256 + (8 << 20)  # A2AV_STATIC_SCRATCH_BYTES
DTYPES = {torch.bfloat16: 0, torch.float16: 1}
PATHS = {"default": 0, "fused": 1, "split": 2, "split_runs": 3}
TILES = {"default": 0, "single": 1, "pair": 2, "pair_k64": 3}

# Every function the headers under include/ declare.
EXPORTS = ("a2av_gmm_workspace_size", "a2av_gmm_run", "a2av_gmm_read_device_status",
           "a2av_gmm_status_string", "a2av_gmm_launch_count", "a2av_gmm_run_static_scratch",
           "a2av_gmm_run_profiled", "a2av_gmm_run_arrivals",
           "a2av_amp_update_scale", "a2av_found_nonfinite", "a2av_quant_reduce",
           "a2av_gmm_mx_workspace_size", "a2av_gmm_mx_run", "a2av_gmm_mx_run_profiled",
           "a2av_rms_norm", "a2av_rms_norm_backward", "a2av_rms_norm_backward_workspace_size", "a2av_glu_quant",
           "a2av_gated_workspace_size", "a2av_gated_run", "a2av_gated_backward",
           "a2av_gmm_backward_workspace_size", "a2av_gmm_backward",
           "a2av_layer_norm", "a2av_layer_norm_backward", "a2av_layer_norm_backward_workspace_size",
           "a2av_gmm_g128_workspace_size", "a2av_gmm_g128_run", "a2av_moe_workspace_size", "a2av_moe_run")
_FFN_EXPORTS = EXPORTS[EXPORTS.index("a2av_rms_norm"):]

# a2av_qtype / a2av_qmode of include/a2av_quant_reduce.h.
QTYPES = {"e4m3fn": 0, "e5m2": 1, "int8": 2}
QMODES = {"mx": 0, "group128": 1}
ACTS = {"silu": 0, "gelu_tanh": 1}  # a2av_act of include/a2av_ffn.h
SCORES = {"softmax": 0, "sigmoid": 1}  # a2av_score of include/a2av_moe.h


class A2avError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class Desc(ctypes.Structure):
    _fields_ = [("W", ctypes.c_int32), ("e", ctypes.c_int32),
                ("A", ctypes.c_int64), ("H1", ctypes.c_int64), ("N1", ctypes.c_int64),
                ("BS", ctypes.c_int64), ("H2", ctypes.c_int64), ("N2", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("want_permute_out", ctypes.c_int32),
                ("path", ctypes.c_int32), ("tiles", ctypes.c_int32)]


class MxDesc(ctypes.Structure):
    """a2av_gmm_mx_desc of include/a2av_gmm_mx.h."""
    _fields_ = [("W", ctypes.c_int32), ("e", ctypes.c_int32),
                ("A", ctypes.c_int64), ("H1", ctypes.c_int64), ("N1", ctypes.c_int64),
                ("BS", ctypes.c_int64), ("H2", ctypes.c_int64), ("N2", ctypes.c_int64),
                ("qtype", ctypes.c_int32), ("want_permute_out", ctypes.c_int32), ("tiles", ctypes.c_int32)]


class RmsNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("H", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64), ("dtype", ctypes.c_int32), ("qtype", ctypes.c_int32),
                ("qmode", ctypes.c_int32), ("eps", ctypes.c_float)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = RmsNormDesc._fields_


class GluDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("N", ctypes.c_int64), ("stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("qtype", ctypes.c_int32),
                ("qmode", ctypes.c_int32)]


class GatedDesc(ctypes.Structure):
    _fields_ = [("W", ctypes.c_int32), ("e", ctypes.c_int32),
                ("A", ctypes.c_int64), ("H1", ctypes.c_int64), ("N", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("want_permute_out", ctypes.c_int32),
                ("save", ctypes.c_int32)]


class G128Desc(ctypes.Structure):
    """a2av_gmm_g128_desc of include/a2av_gmm_g128.h."""
    _fields_ = [("W", ctypes.c_int32), ("e", ctypes.c_int32),
                ("A", ctypes.c_int64), ("H1", ctypes.c_int64), ("N1", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("qtype", ctypes.c_int32)]


class MoeDesc(ctypes.Structure):
    """a2av_moe_desc of include/a2av_moe.h."""
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("K", ctypes.c_int32),
                ("H", ctypes.c_int64), ("N", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("router_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("score", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None


def lib_path() -> str:
    return _build.LIB


def load():
    """Load the built library (raises if it was not built)."""
    global _lib
    if _lib is None:
        _lib = load_library(_build.LIB)
    return _lib


def load_checks():
    """The debug build with device-side bounds checks (built by build.build(checks=True)),
    as a separate handle with the same functions."""
    return load_library(_build.CHECKS_LIB)


def load_library(path: str):
    """Open one build of the library and declare every C-ABI function's signature."""
    if not os.path.exists(path):
        raise ImportError(f"CUDA library not built: {path} (run __graft_entry__.build())")
    L = ctypes.CDLL(path)
    p, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    L.a2av_gmm_workspace_size.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(sz)]
    L.a2av_gmm_workspace_size.restype = ctypes.c_int
    L.a2av_gmm_run.argtypes = [ctypes.POINTER(Desc), p, p, p, p, p, p, p, p, p, sz, p]
    L.a2av_gmm_run.restype = ctypes.c_int
    L.a2av_gmm_run_profiled.argtypes = [ctypes.POINTER(Desc), p, p, p, p, p, p, p, p, p, sz, p, p, p]
    L.a2av_gmm_run_profiled.restype = ctypes.c_int
    L.a2av_gmm_run_arrivals.argtypes = [ctypes.POINTER(Desc), p, p, p, p, p, p, p, p, p, ctypes.c_uint64,
                                        ctypes.c_uint64, p, sz, p]
    L.a2av_gmm_run_arrivals.restype = ctypes.c_int
    L.a2av_gmm_read_device_status.argtypes = [p, p, ctypes.POINTER(i32)]
    L.a2av_gmm_read_device_status.restype = ctypes.c_int
    L.a2av_gmm_status_string.argtypes = [ctypes.c_int]
    L.a2av_gmm_status_string.restype = ctypes.c_char_p
    L.a2av_gmm_launch_count.argtypes = [ctypes.POINTER(Desc)]
    L.a2av_gmm_launch_count.restype = i32
    L.a2av_gmm_run_static_scratch.argtypes = [ctypes.POINTER(Desc), p, p, p, p, p, p, p, p, p]
    L.a2av_gmm_run_static_scratch.restype = ctypes.c_int
    L.a2av_amp_update_scale.argtypes = [p, p, p, ctypes.c_float, ctypes.c_float, i32, p]
    L.a2av_amp_update_scale.restype = ctypes.c_int
    L.a2av_found_nonfinite.argtypes = [p, ctypes.c_int64, i32, p, p]
    L.a2av_found_nonfinite.restype = ctypes.c_int
    L.a2av_quant_reduce.argtypes = [i32, ctypes.c_int64, ctypes.c_int64, i32, i32, p, p, p, i32, p]
    L.a2av_quant_reduce.restype = ctypes.c_int
    L.a2av_gmm_mx_workspace_size.argtypes = [ctypes.POINTER(MxDesc), ctypes.POINTER(sz)]
    L.a2av_gmm_mx_workspace_size.restype = ctypes.c_int
    L.a2av_gmm_mx_run.argtypes = [ctypes.POINTER(MxDesc)] + [p] * 14 + [sz, p]
    L.a2av_gmm_mx_run.restype = ctypes.c_int
    L.a2av_gmm_mx_run_profiled.argtypes = [ctypes.POINTER(MxDesc)] + [p] * 14 + [sz, p, p, p]
    L.a2av_gmm_mx_run_profiled.restype = ctypes.c_int
    i64, psz = ctypes.c_int64, ctypes.POINTER(sz)
    L.a2av_rms_norm.argtypes = [ctypes.POINTER(RmsNormDesc)] + [p] * 9
    L.a2av_rms_norm_backward_workspace_size.argtypes = [i64, i64, i32, psz]
    L.a2av_rms_norm_backward.argtypes = [i64, i64, i32] + [p] * 8 + [sz, p]
    L.a2av_glu_quant.argtypes = [ctypes.POINTER(GluDesc)] + [p] * 6
    L.a2av_gated_workspace_size.argtypes = [ctypes.POINTER(GatedDesc), psz]
    L.a2av_gated_run.argtypes = [ctypes.POINTER(GatedDesc)] + [p] * 8 + [sz, p]
    L.a2av_gated_backward.argtypes = [ctypes.POINTER(GatedDesc)] + [p] * 10 + [sz, p]
    L.a2av_gmm_backward_workspace_size.argtypes = [ctypes.POINTER(Desc), psz]
    L.a2av_gmm_backward.argtypes = [ctypes.POINTER(Desc)] + [p] * 7 + [sz, p]
    L.a2av_layer_norm.argtypes = [ctypes.POINTER(LayerNormDesc)] + [p] * 11
    L.a2av_layer_norm_backward_workspace_size.argtypes = [i64, i64, i32, psz]
    L.a2av_layer_norm_backward.argtypes = [i64, i64, i32] + [p] * 10 + [sz, p]
    L.a2av_gmm_g128_workspace_size.argtypes = [ctypes.POINTER(G128Desc), psz]
    L.a2av_gmm_g128_run.argtypes = [ctypes.POINTER(G128Desc)] + [p] * 7 + [sz, p]
    L.a2av_moe_workspace_size.argtypes = [ctypes.POINTER(MoeDesc), psz]
    L.a2av_moe_run.argtypes = [ctypes.POINTER(MoeDesc)] + [p] * 11 + [sz, p]
    for name in _FFN_EXPORTS:
        getattr(L, name).restype = ctypes.c_int
    return L


def make_desc(W, e, A, H1, N1, BS=0, H2=0, N2=0, dtype=torch.bfloat16, want_permute_out=False,
              path="default", tiles="default") -> Desc:
    return Desc(W, e, A, H1, N1, BS, H2, N2, DTYPES[dtype], int(bool(want_permute_out)), PATHS[path],
                TILES[tiles])


def a2av_gmm_workspace_size(desc: Desc) -> int:
    n = ctypes.c_size_t(0)
    st = load().a2av_gmm_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if st != A2AV_OK:
        raise A2avError(st, "a2av_gmm_workspace_size")
    return n.value


def a2av_gmm_launch_count(desc: Desc) -> int:
    return int(load().a2av_gmm_launch_count(ctypes.byref(desc)))


def a2av_gmm_status_string(status: int) -> str:
    return load().a2av_gmm_status_string(status).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def a2av_gmm_run(desc: Desc, ataOut, recvCounts, gmmWeight, mmX, mmWeight, permuteOut, gmmY, mmY,
                 workspace: torch.Tensor, stream=None) -> None:
    """Raw phase 2: device tensors (or None) in, enqueued on the stream."""
    s = stream if stream is not None else torch.cuda.current_stream()
    st = load().a2av_gmm_run(ctypes.byref(desc), _ptr(ataOut), _ptr(recvCounts), _ptr(gmmWeight),
                             _ptr(mmX), _ptr(mmWeight), _ptr(permuteOut), _ptr(gmmY), _ptr(mmY),
                             _ptr(workspace), workspace.numel(), ctypes.c_void_p(s.cuda_stream))
    if st != A2AV_OK:
        raise A2avError(st, "a2av_gmm_run")


def a2av_gmm_run_profiled(desc: Desc, ataOut, recvCounts, gmmWeight, mmX, mmWeight, permuteOut, gmmY, mmY,
                          workspace: torch.Tensor, gemm_begin: torch.cuda.Event, gemm_end: torch.cuda.Event,
                          stream=None) -> None:
    """a2av_gmm_run with two timing events (torch.cuda.Event(enable_timing=True)) recorded
    right before and after the grouped-GEMM kernel."""
    s = stream if stream is not None else torch.cuda.current_stream()
    for ev in (gemm_begin, gemm_end):
        if ev.cuda_event == 0:  # created lazily by torch: make it exist on this device
            ev.record(s)
    st = load().a2av_gmm_run_profiled(ctypes.byref(desc), _ptr(ataOut), _ptr(recvCounts), _ptr(gmmWeight),
                                      _ptr(mmX), _ptr(mmWeight), _ptr(permuteOut), _ptr(gmmY), _ptr(mmY),
                                      _ptr(workspace), workspace.numel(), ctypes.c_void_p(s.cuda_stream),
                                      ctypes.c_void_p(gemm_begin.cuda_event), ctypes.c_void_p(gemm_end.cuda_event))
    if st != A2AV_OK:
        raise A2avError(st, "a2av_gmm_run_profiled")


def a2av_gmm_run_arrivals(desc: Desc, ataOut, recvCounts, gmmWeight, mmX, mmWeight, permuteOut, gmmY, mmY,
                          arrived: torch.Tensor, arrival_tag: int, wait_limit_ns: int, workspace: torch.Tensor,
                          stream=None) -> None:
    """a2av_gmm_run that starts before the rows have all arrived: source w's rows of ataOut are
    read once arrived[w] (an int64 device tensor of W flags) equals arrival_tag."""
    _check(arrived, "arrived", torch.int64, 1)
    s = stream if stream is not None else torch.cuda.current_stream()
    st = load().a2av_gmm_run_arrivals(ctypes.byref(desc), _ptr(ataOut), _ptr(recvCounts), _ptr(gmmWeight),
                                      _ptr(mmX), _ptr(mmWeight), _ptr(permuteOut), _ptr(gmmY), _ptr(mmY),
                                      _ptr(arrived), ctypes.c_uint64(arrival_tag & (2**64 - 1)),
                                      ctypes.c_uint64(wait_limit_ns), _ptr(workspace), workspace.numel(),
                                      ctypes.c_void_p(s.cuda_stream))
    if st != A2AV_OK:
        raise A2avError(st, "a2av_gmm_run_arrivals")


def a2av_gmm_run_static_scratch(desc: Desc, ataOut, recvCounts, gmmWeight, mmX, mmWeight, permuteOut, gmmY,
                                mmY, stream=None) -> int:
    """Phase 2 without a workspace, for callers that cannot allocate device
    memory: the library's own static device scratch array stands in for it.
    Returns the status code (0 = enqueued)."""
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(load().a2av_gmm_run_static_scratch(
        ctypes.byref(desc), _ptr(ataOut), _ptr(recvCounts), _ptr(gmmWeight), _ptr(mmX), _ptr(mmWeight),
        _ptr(permuteOut), _ptr(gmmY), _ptr(mmY), ctypes.c_void_p(s.cuda_stream)))


def a2av_amp_update_scale(scale: torch.Tensor, growth_tracker: torch.Tensor, found_inf: torch.Tensor,
                          growth_factor: float, backoff_factor: float, growth_interval: int, stream=None) -> None:
    """In place on device scalars: scale (float32 [1]), growth_tracker (int32 [1]), found_inf (float32 [1])."""
    _check(scale, "scale", torch.float32)
    _check(growth_tracker, "growth_tracker", torch.int32)
    _check(found_inf, "found_inf", torch.float32)
    s = stream if stream is not None else torch.cuda.current_stream()
    st = load().a2av_amp_update_scale(_ptr(scale), _ptr(growth_tracker), _ptr(found_inf), growth_factor,
                                      backoff_factor, growth_interval, ctypes.c_void_p(s.cuda_stream))
    if st != A2AV_OK:
        raise A2avError(st, "a2av_amp_update_scale")


def a2av_found_nonfinite(x: torch.Tensor, found_inf: torch.Tensor, stream=None) -> None:
    """found_inf (float32 [1], device) = 1 when x holds an inf or NaN; unchanged otherwise."""
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[x.dtype]
    _check(x, "x")
    _check(found_inf, "found_inf", torch.float32)
    s = stream if stream is not None else torch.cuda.current_stream()
    st = load().a2av_found_nonfinite(_ptr(x) if x.numel() else None, x.numel(), code, _ptr(found_inf),
                                     ctypes.c_void_p(s.cuda_stream))
    if st != A2AV_OK:
        raise A2avError(st, "a2av_found_nonfinite")


def a2av_quant_reduce(data: torch.Tensor, scales: torch.Tensor, qtype: str, mode: str,
                      out: torch.Tensor, stream=None) -> torch.Tensor:
    """out [rows, H] = sum over w of decode(data[w]) * scales[w] ("aclnnQuantReduceScatter" page,
    Formula).  data: uint8 [W, rows, H] codes of qtype ("e4m3fn", "e5m2", "int8"); scales: uint8
    E8M0 [W, rows, H/32] for mode "mx", float32 [W, rows, H/128] for "group128"; out: bf16, fp16
    or fp32 [rows, H]."""
    _check(data, "data", torch.uint8, 3)
    _check(scales, "scales", torch.uint8 if mode == "mx" else torch.float32, 3)
    _check(out, "out", None, 2)
    W, rows, H = data.shape
    if tuple(out.shape) != (rows, H):
        raise ValueError(f"out must be [{rows}, {H}], got {tuple(out.shape)}")
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[out.dtype]
    s = stream if stream is not None else torch.cuda.current_stream()
    st = load().a2av_quant_reduce(W, rows, H, QTYPES[qtype], QMODES[mode], _ptr(data), _ptr(scales),
                                  _ptr(out), code, ctypes.c_void_p(s.cuda_stream))
    if st != A2AV_OK:
        raise A2avError(st, "a2av_quant_reduce")
    return out


def a2av_gmm_read_device_status(workspace: torch.Tensor, stream=None) -> tuple[int, int]:
    s = stream if stream is not None else torch.cuda.current_stream()
    code = ctypes.c_int32(0)
    st = load().a2av_gmm_read_device_status(_ptr(workspace), ctypes.c_void_p(s.cuda_stream),
                                             ctypes.byref(code))
    return st, code.value


def _check(t, name, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


class Plan:
    """Descriptor + workspace for one shape, reusable across calls."""

    def __init__(self, W, e, A, H1, N1, BS=0, H2=0, N2=0, dtype=torch.bfloat16,
                 want_permute_out=False, path="default", device=None, tiles="default"):
        self.desc = make_desc(W, e, A, H1, N1, BS, H2, N2, dtype, want_permute_out, path, tiles)
        self.dtype = dtype
        self.device = torch.device(device) if device is not None else torch.device("cuda")
        self.workspace = torch.empty(a2av_gmm_workspace_size(self.desc), dtype=torch.uint8, device=self.device)

    def run(self, ataOut, recvCounts, gmmWeight, mmX=None, mmWeight=None, gmmY=None, mmY=None,
            permuteOut=None, stream=None, gemm_events=None):
        """gemm_events: optional (begin, end) timing events recorded around the GEMM kernel
        (a2av_gmm_run_profiled)."""
        d = self.desc
        if d.A:
            _check(ataOut, "ataOut", self.dtype, 2)
        _check(recvCounts, "recvCounts", torch.int32, 1)
        _check(gmmWeight, "gmmWeight", self.dtype, 3)
        if tuple(gmmWeight.shape) != (d.e, d.H1, d.N1):
            raise ValueError("gmmWeight shape")
        if recvCounts.numel() != d.W * d.e:
            raise ValueError("recvCounts length")
        if gmmY is None:
            gmmY = torch.empty(d.A, d.N1, dtype=self.dtype, device=self.device)
        if d.want_permute_out and permuteOut is None:
            permuteOut = torch.empty(d.A, d.H1, dtype=self.dtype, device=self.device)
        if d.BS:
            _check(mmX, "mmX", self.dtype, 2)
            _check(mmWeight, "mmWeight", self.dtype, 2)
            if mmY is None:
                mmY = torch.empty(d.BS, d.N2, dtype=self.dtype, device=self.device)
        args = (d, ataOut if d.A else None, recvCounts, gmmWeight, mmX, mmWeight,
                permuteOut if d.want_permute_out else None, gmmY if d.A else None,
                mmY if d.BS else None, self.workspace)
        if gemm_events is None:
            a2av_gmm_run(*args, stream)
        else:
            a2av_gmm_run_profiled(*args, gemm_events[0], gemm_events[1], stream)
        return gmmY, mmY, permuteOut


def a2av_gmm(ataOut, recvCounts, gmmWeight, mmX=None, mmWeight=None, return_permute=False,
             W=None, path="default", tiles="default"):
    """permuteOut = Permute(ataOut); gmmY = permuteOut x gmmWeight; mmY = mmX x mmWeight.

    Returns (gmmY, mmY or None, permuteOut or None).  W defaults to
    len(recvCounts) // e.
    """
    e, H1, N1 = gmmWeight.shape
    if W is None:
        W = recvCounts.numel() // e
    BS, H2, N2 = (0, 0, 0)
    if mmX is not None:
        BS, H2 = mmX.shape
        N2 = mmWeight.shape[1]
    plan = Plan(W, e, ataOut.shape[0], H1, N1, BS, H2, N2, gmmWeight.dtype, return_permute, path,
                device=gmmWeight.device, tiles=tiles)
    return plan.run(ataOut, recvCounts, gmmWeight, mmX, mmWeight)


class MxPlan:
    """Descriptor + workspace of the block-scaled FP8 (mx) call for one shape
    (include/a2av_gmm_mx.h): codes as uint8 tensors, E8M0 scales as uint8
    tensors with one byte per 32 codes along K, weights [e, N1, H1]."""

    def __init__(self, W, e, A, H1, N1, BS=0, H2=0, N2=0, qtype="e4m3fn", want_permute_out=False, device=None,
                 tiles="default"):
        self.desc = MxDesc(W, e, A, H1, N1, BS, H2, N2, QTYPES[qtype], int(bool(want_permute_out)), TILES[tiles])
        self.device = torch.device(device) if device is not None else torch.device("cuda")
        n = ctypes.c_size_t(0)
        st = load().a2av_gmm_mx_workspace_size(ctypes.byref(self.desc), ctypes.byref(n))
        if st != A2AV_OK:
            raise A2avError(st, "a2av_gmm_mx_workspace_size")
        self.workspace = torch.empty(n.value, dtype=torch.uint8, device=self.device)

    def run(self, ataOut_q, ataOut_s, recvCounts, gmmWeight_q, gmmWeight_s, mmX_q=None, mmX_s=None,
            mmWeight_q=None, mmWeight_s=None, gmmY=None, mmY=None, permuteOut_q=None, permuteOut_s=None,
            stream=None, gemm_events=None):
        """Returns (gmmY, mmY, permuteOut_q, permuteOut_s); outputs are bf16.
        gemm_events: optional (begin, end) timing events recorded around the
        GEMM kernel (a2av_gmm_mx_run_profiled)."""
        d = self.desc
        for t, name in ((ataOut_q, "ataOut_q"), (ataOut_s, "ataOut_s")):
            if d.A:
                _check(t, name, torch.uint8, 2)
        _check(recvCounts, "recvCounts", torch.int32, 1)
        _check(gmmWeight_q, "gmmWeight_q", torch.uint8, 3)
        _check(gmmWeight_s, "gmmWeight_s", torch.uint8, 3)
        if tuple(gmmWeight_q.shape) != (d.e, d.N1, d.H1) or tuple(gmmWeight_s.shape) != (d.e, d.N1, d.H1 // 32):
            raise ValueError("gmmWeight_q must be [e, N1, H1] and gmmWeight_s [e, N1, H1/32]")
        if d.A and (tuple(ataOut_q.shape) != (d.A, d.H1) or tuple(ataOut_s.shape) != (d.A, d.H1 // 32)):
            raise ValueError("ataOut_q must be [A, H1] and ataOut_s [A, H1/32]")
        if gmmY is None:
            gmmY = torch.empty(d.A, d.N1, dtype=torch.bfloat16, device=self.device)
        if d.want_permute_out:
            if permuteOut_q is None:
                permuteOut_q = torch.empty(d.A, d.H1, dtype=torch.uint8, device=self.device)
            if permuteOut_s is None:
                permuteOut_s = torch.empty(d.A, d.H1 // 32, dtype=torch.uint8, device=self.device)
        if d.BS:
            for t, name in ((mmX_q, "mmX_q"), (mmX_s, "mmX_s"), (mmWeight_q, "mmWeight_q"),
                            (mmWeight_s, "mmWeight_s")):
                _check(t, name, torch.uint8, 2)
            if mmY is None:
                mmY = torch.empty(d.BS, d.N2, dtype=torch.bfloat16, device=self.device)
        s = stream if stream is not None else torch.cuda.current_stream()
        args = (ctypes.byref(d), _ptr(ataOut_q) if d.A else None, _ptr(ataOut_s) if d.A else None,
                _ptr(recvCounts), _ptr(gmmWeight_q), _ptr(gmmWeight_s), _ptr(mmX_q) if d.BS else None,
                _ptr(mmX_s) if d.BS else None, _ptr(mmWeight_q) if d.BS else None,
                _ptr(mmWeight_s) if d.BS else None, _ptr(permuteOut_q) if d.want_permute_out else None,
                _ptr(permuteOut_s) if d.want_permute_out else None, _ptr(gmmY) if d.A else None,
                _ptr(mmY) if d.BS else None, _ptr(self.workspace), self.workspace.numel(),
                ctypes.c_void_p(s.cuda_stream))
        if gemm_events is None:
            name = "a2av_gmm_mx_run"
            st = load().a2av_gmm_mx_run(*args)
        else:
            name = "a2av_gmm_mx_run_profiled"
            for ev in gemm_events:
                if ev.cuda_event == 0:  # created lazily by torch: make it exist on this device
                    ev.record(s)
            st = load().a2av_gmm_mx_run_profiled(*args, ctypes.c_void_p(gemm_events[0].cuda_event),
                                                 ctypes.c_void_p(gemm_events[1].cuda_event))
        if st != A2AV_OK:
            raise A2avError(st, name)
        return gmmY, mmY, permuteOut_q, permuteOut_s


# ---- the operators around the grouped product (include/a2av_ffn.h)


# These calls are a few microseconds on the GPU for a single token, so their checks are kept to the fewest steps.


def _call(name, *args):
    st = getattr(_lib or load(), name)(*args)
    if st != A2AV_OK:
        raise A2avError(st, name)


def _size(name, *args) -> int:
    n = ctypes.c_size_t(0)
    _call(name, *args, ctypes.byref(n))
    return n.value


def _at(t):
    return None if t is None else t.data_ptr()


_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # of a device, as a handle


def _enqueue(name, device, stream, *args):
    """The call `name` on the given stream, or the current one of this device, which is the current device meanwhile: the
    library asks it for its limits."""
    if stream is None:
        handle = _current_stream(device)
    elif stream.device_index == device:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"stream must be of cuda:{device}, got one of cuda:{stream.device_index}")
    if _current_device() != device:
        with torch.cuda.device(device):
            return _enqueue(name, device, stream, *args)
    _call(name, *args, handle)


def _beside(t, name, device):
    """Refuses a tensor of another device."""
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got cuda:{t.get_device()}")


def _is(t, name, dtype, shape, device):
    """t is a contiguous CUDA tensor of this type and shape on this device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        _beside(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows_of(t, name):
    """A 2-D CUDA tensor of 16-bit floats whose rows are contiguous; returns (type code, elements from one row to the
    next)."""
    code = DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor, got {getattr(t, 'dtype', type(t))}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions")
    rows, cols = t.shape
    step, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return code, step if rows > 1 else cols


def _out(t, name, dtype, shape, like, stream):
    """The caller's output tensor, checked, or a new one on `like`'s device, of the stream that writes it."""
    if t is None:
        if stream is not None:
            with torch.cuda.stream(stream):
                return torch.empty(shape, dtype=dtype, device=like.device)
        if like.shape == shape and like.dtype == dtype and like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=like.device)
    _is(t, name, dtype, shape, like.get_device())
    return t


def _named(table, key, what):
    if key not in table:
        raise ValueError(f"{what} must be one of {sorted(table)}, got {key!r}")
    return table[key]


def _code_outputs(out, rows, cols, mode, like, stream):
    """(codes, scales) to write: those of an earlier result, or new ones."""
    mx = mode == "mx"
    return (_out(out.codes if out else None, "codes", torch.uint8, (rows, cols), like, stream),
            _out(out.scales if out else None, "scales", torch.uint8 if mx else torch.float32,
                 (rows, cols // (32 if mx else 128)), like, stream))


class _RmsNormFields(NamedTuple):
    h: Optional[torch.Tensor]       # x + residual, element type (None without a residual)
    y: Optional[torch.Tensor]       # normed rows, element type
    codes: Optional[torch.Tensor]   # uint8 codes of the normed rows
    scales: Optional[torch.Tensor]  # uint8 E8M0 per 32 (mx) or float32 per 128 (group128)
    rstd: Optional[torch.Tensor]    # float32 [rows]


class RmsNormOut(_RmsNormFields):
    """Also holds, for a call that writes its tensors again, what they were made for and the descriptor."""


def a2av_rms_norm(x, gamma, residual=None, eps=1e-6, qtype=None, mode="mx", want_y=None, want_rstd=False,
                  out: Optional[RmsNormOut] = None, stream=None) -> RmsNormOut:
    """RMS norm of x [rows, H] (+ residual), times gamma [H]: the normed rows as codes and scales (qtype "e4m3fn",
    "e5m2" or "int8"; mode "mx" or "group128") and / or in the element type (want_y; by default without a qtype).
    Rows of x and residual may be strided; residual may be one row expanded to all.  `out`: an earlier result of the
    same call, whose tensors are written again."""
    code, xs = _rows_of(x, "x")
    shape, dtype, device = x.shape, x.dtype, x.get_device()
    rows, H = shape
    _is(gamma, "gamma", dtype, (H,), device)
    rs = None
    if residual is not None:
        _, rs = _rows_of(residual, "residual")
        if residual.shape != shape or residual.dtype != dtype:
            raise ValueError("residual must have the shape and type of x")
        if residual.get_device() != device:
            _beside(residual, "residual", device)
    key = (shape, dtype, xs, rs, eps, qtype, mode, want_y, want_rstd, device)
    if out is not None and getattr(out, "key", None) == key:  # its tensors and descriptor fit as they are
        h, y, codes, scales, rstd = out
        _enqueue("a2av_rms_norm", device, stream, out.desc, x.data_ptr(), _at(residual), gamma.data_ptr(), _at(h), _at(y),
                 _at(codes), _at(scales), _at(rstd))
        return out
    q, m = -1 if qtype is None else _named(QTYPES, qtype, "qtype"), _named(QMODES, mode, "mode")
    h = None if residual is None else _out(out.h if out else None, "h", dtype, shape, x, stream)
    y = codes = scales = rstd = None
    if want_y or (want_y is None and qtype is None):
        y = _out(out.y if out else None, "y", dtype, shape, x, stream)
    if want_rstd:
        rstd = _out(out.rstd if out else None, "rstd", torch.float32, (rows,), x, stream)
    if qtype is not None:
        codes, scales = _code_outputs(out, rows, H, mode, x, stream)
    desc = ctypes.byref(RmsNormDesc(rows, H, xs, rs or 0, code, q, m, eps))
    _enqueue("a2av_rms_norm", device, stream, desc, x.data_ptr(), _at(residual), gamma.data_ptr(), _at(h), _at(y),
             _at(codes), _at(scales), _at(rstd))
    result = RmsNormOut(h, y, codes, scales, rstd)
    result.key, result.desc = key, desc
    return result


@functools.lru_cache(maxsize=256)
def _norm_backward_size(rows, H, code):
    return _size("a2av_rms_norm_backward_workspace_size", rows, H, code)


def a2av_rms_norm_backward(dy, h, gamma, rstd, dh=None, dx=None, dgamma=None, workspace=None, stream=None):
    """(dx [rows, H], dgamma float32 [H]) from the gradient dy of the normed rows and, optionally, the gradient dh
    that reaches h directly.  dx is the gradient of x and of the residual."""
    code, _ = _rows_of(dy, "dy")
    shape, dtype, device = dy.shape, dy.dtype, dy.get_device()
    rows, H = shape
    _is(dy, "dy", dtype, shape, device)
    _is(h, "h", dtype, shape, device)
    if dh is not None:
        _is(dh, "dh", dtype, shape, device)
    _is(gamma, "gamma", dtype, (H,), device)
    _is(rstd, "rstd", torch.float32, (rows,), device)
    dx = _out(dx, "dx", dtype, shape, dy, stream)
    dgamma = _out(dgamma, "dgamma", torch.float32, (H,), dy, stream)
    need = _norm_backward_size(rows, H, code)
    if workspace is None and need:
        workspace = _out(None, "workspace", torch.uint8, (need,), dy, stream)
    elif workspace is not None:
        _beside(workspace, "workspace", device)
    _enqueue("a2av_rms_norm_backward", device, stream, rows, H, code, _at(dy), _at(dh), _at(h), _at(gamma), _at(rstd),
             _at(dx), _at(dgamma), _at(workspace), 0 if workspace is None else workspace.numel())
    return dx, dgamma


class _LayerNormFields(NamedTuple):
    h: Optional[torch.Tensor]       # x + residual, element type (None without a residual)
    y: Optional[torch.Tensor]       # normed rows, element type
    codes: Optional[torch.Tensor]   # uint8 codes of the normed rows
    scales: Optional[torch.Tensor]  # uint8 E8M0 per 32 (mx) or float32 per 128 (group128)
    mean: Optional[torch.Tensor]    # float32 [rows]
    rstd: Optional[torch.Tensor]    # float32 [rows]


class LayerNormOut(_LayerNormFields):
    """Also holds what its tensors were made for and the descriptor, as RmsNormOut does."""


def a2av_layer_norm(x, gamma, beta=None, residual=None, eps=1e-5, qtype=None, mode="mx", want_y=None, want_stats=False,
                    out: Optional[LayerNormOut] = None, stream=None) -> LayerNormOut:
    """Layer norm of x [rows, H] (+ residual), times gamma [H], plus beta [H] where given: the normed rows as codes and
    scales (qtype "e4m3fn", "e5m2" or "int8"; mode "mx" or "group128") and / or in the element type (want_y; by default
    without a qtype).  want_stats: mean and rstd too, for the backward pass.  Rows of x and residual may be strided;
    residual may be one row expanded to all.  `out`: an earlier result of the same call, whose tensors are written
    again."""
    code, xs = _rows_of(x, "x")
    shape, dtype, device = x.shape, x.dtype, x.get_device()
    rows, H = shape
    _is(gamma, "gamma", dtype, (H,), device)
    if beta is not None:
        _is(beta, "beta", dtype, (H,), device)
    rs = None
    if residual is not None:
        _, rs = _rows_of(residual, "residual")
        if residual.shape != shape or residual.dtype != dtype:
            raise ValueError("residual must have the shape and type of x")
        if residual.get_device() != device:
            _beside(residual, "residual", device)
    key = (shape, dtype, xs, rs, eps, qtype, mode, want_y, want_stats, device)
    if out is not None and getattr(out, "key", None) == key:  # its tensors and descriptor fit as they are
        h, y, codes, scales, mean, rstd = out
        _enqueue("a2av_layer_norm", device, stream, out.desc, x.data_ptr(), _at(residual), gamma.data_ptr(), _at(beta),
                 _at(h), _at(y), _at(codes), _at(scales), _at(mean), _at(rstd))
        return out
    q, m = -1 if qtype is None else _named(QTYPES, qtype, "qtype"), _named(QMODES, mode, "mode")
    h = None if residual is None else _out(out.h if out else None, "h", dtype, shape, x, stream)
    y = codes = scales = mean = rstd = None
    if want_y or (want_y is None and qtype is None):
        y = _out(out.y if out else None, "y", dtype, shape, x, stream)
    if want_stats:
        mean = _out(out.mean if out else None, "mean", torch.float32, (rows,), x, stream)
        rstd = _out(out.rstd if out else None, "rstd", torch.float32, (rows,), x, stream)
    if qtype is not None:
        codes, scales = _code_outputs(out, rows, H, mode, x, stream)
    desc = ctypes.byref(LayerNormDesc(rows, H, xs, rs or 0, code, q, m, eps))
    _enqueue("a2av_layer_norm", device, stream, desc, x.data_ptr(), _at(residual), gamma.data_ptr(), _at(beta), _at(h),
             _at(y), _at(codes), _at(scales), _at(mean), _at(rstd))
    result = LayerNormOut(h, y, codes, scales, mean, rstd)
    result.key, result.desc = key, desc
    return result


@functools.lru_cache(maxsize=256)
def _layer_norm_backward_size(rows, H, code):
    return _size("a2av_layer_norm_backward_workspace_size", rows, H, code)


def a2av_layer_norm_backward(dy, h, gamma, mean, rstd, dh=None, dx=None, dgamma=None, dbeta=None, workspace=None,
                             stream=None):
    """(dx [rows, H], dgamma float32 [H], dbeta float32 [H]) from the gradient dy of the normed rows and, optionally,
    the gradient dh that reaches h directly.  dx is the gradient of x and of the residual."""
    code, _ = _rows_of(dy, "dy")
    shape, dtype, device = dy.shape, dy.dtype, dy.get_device()
    rows, H = shape
    _is(dy, "dy", dtype, shape, device)
    _is(h, "h", dtype, shape, device)
    if dh is not None:
        _is(dh, "dh", dtype, shape, device)
    _is(gamma, "gamma", dtype, (H,), device)
    _is(mean, "mean", torch.float32, (rows,), device)
    _is(rstd, "rstd", torch.float32, (rows,), device)
    dx = _out(dx, "dx", dtype, shape, dy, stream)
    dgamma = _out(dgamma, "dgamma", torch.float32, (H,), dy, stream)
    dbeta = _out(dbeta, "dbeta", torch.float32, (H,), dy, stream)
    need = _layer_norm_backward_size(rows, H, code)
    if workspace is None and need:
        workspace = _out(None, "workspace", torch.uint8, (need,), dy, stream)
    elif workspace is not None:
        _beside(workspace, "workspace", device)
    _enqueue("a2av_layer_norm_backward", device, stream, rows, H, code, _at(dy), _at(dh), _at(h), _at(gamma), _at(mean),
             _at(rstd), _at(dx), _at(dgamma), _at(dbeta), _at(workspace), 0 if workspace is None else workspace.numel())
    return dx, dgamma, dbeta


class _GluQuantFields(NamedTuple):
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    h: Optional[torch.Tensor]


class GluQuantOut(_GluQuantFields):
    """Also holds what its tensors were made for and the descriptor, as RmsNormOut does."""


def a2av_glu_quant(gate_up, act="silu", qtype="e4m3fn", mode="mx", want_h=None, out: Optional[GluQuantOut] = None,
                   stream=None) -> GluQuantOut:
    """act(gate) * up of gate_up [rows, 2N] (gate columns, then up columns) as codes and scales and / or in the
    element type (want_h; by default without a qtype)."""
    code, stride = _rows_of(gate_up, "gate_up")
    shape, device = gate_up.shape, gate_up.get_device()
    rows, cols = shape
    N = cols // 2
    if cols != 2 * N:
        raise ValueError("gate_up must have an even number of columns")
    gate = gate_up.data_ptr()
    key = (shape, gate_up.dtype, stride, act, qtype, mode, want_h, device)
    if out is not None and getattr(out, "key", None) == key:
        codes, scales, h = out
        _enqueue("a2av_glu_quant", device, stream, out.desc, gate, gate + 2 * N if gate else None, _at(h), _at(codes),
                 _at(scales))
        return out
    q = -1 if qtype is None else _named(QTYPES, qtype, "qtype")
    desc = ctypes.byref(GluDesc(rows, N, stride, code, _named(ACTS, act, "act"), q, _named(QMODES, mode, "mode")))
    codes = scales = h = None
    if qtype is not None:
        codes, scales = _code_outputs(out, rows, N, mode, gate_up, stream)
    if want_h or (want_h is None and qtype is None):
        h = _out(out.h if out else None, "h", gate_up.dtype, (rows, N), gate_up, stream)
    _enqueue("a2av_glu_quant", device, stream, desc, gate, gate + 2 * N if gate else None, _at(h), _at(codes), _at(scales))
    result = GluQuantOut(codes, scales, h)
    result.key, result.desc = key, desc
    return result


class GatedOut(NamedTuple):
    h: torch.Tensor                     # [A, N], expert-major
    saved: Optional[torch.Tensor]       # float32 [2, A, N]: gate and up before the activation
    permuteOut: Optional[torch.Tensor]  # expert-major rows (W = 1: ataOut itself)


class GatedGrads(NamedTuple):
    dAtaOut: Optional[torch.Tensor]  # [A, H1], rank-major
    dGate: Optional[torch.Tensor]    # [e, H1, N]
    dUp: Optional[torch.Tensor]      # [e, H1, N]


class GatedPlan:
    """Descriptor + workspace of the gated block h = act(X Wg) * (X Wu) over ragged experts, and its backward pass,
    for one shape.  save: keep what the backward pass needs (with several sources that includes permuteOut).  The
    workspace serves one call at a time: calls of one plan on different streams have to be ordered by the caller."""

    def __init__(self, W, e, A, H1, N, dtype=torch.bfloat16, act="silu", save=False, want_permute_out=None,
                 device=None):
        if want_permute_out is None:
            want_permute_out = save and W > 1
        if dtype not in DTYPES:
            raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
        self.desc = GatedDesc(W, e, A, H1, N, DTYPES[dtype], _named(ACTS, act, "act"), int(bool(want_permute_out)),
                              int(bool(save)))
        self.dtype = dtype
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.workspace = torch.empty(_size("a2av_gated_workspace_size", ctypes.byref(self.desc)), dtype=torch.uint8,
                                     device=self.device)

    def _check_shared(self, recvCounts, gateWeight, upWeight, device):
        d = self.desc
        _is(recvCounts, "recvCounts", torch.int32, (d.W * d.e,), device)
        _is(gateWeight, "gateWeight", self.dtype, (d.e, d.H1, d.N), device)
        _is(upWeight, "upWeight", self.dtype, (d.e, d.H1, d.N), device)

    def run(self, ataOut, recvCounts, gateWeight, upWeight, h=None, saved=None, permuteOut=None,
            stream=None) -> GatedOut:
        d, dtype, ws, device = self.desc, self.dtype, self.workspace, self.workspace.get_device()
        A, H1, N = d.A, d.H1, d.N
        _is(ataOut, "ataOut", dtype, (A, H1), device)
        self._check_shared(recvCounts, gateWeight, upWeight, device)
        h = _out(h, "h", dtype, (A, N), ws, stream)
        saved = _out(saved, "saved", torch.float32, (2, A, N), ws, stream) if d.save else None
        permuted = _out(permuteOut, "permuteOut", dtype, (A, H1), ataOut, stream) if d.want_permute_out else None
        _enqueue("a2av_gated_run", device, stream, ctypes.byref(d), ataOut.data_ptr(), recvCounts.data_ptr(),
                 gateWeight.data_ptr(), upWeight.data_ptr(), _at(permuted), h.data_ptr(), _at(saved), ws.data_ptr(),
                 ws.numel())
        return GatedOut(h, saved, ataOut if d.W == 1 else permuted)

    def backward(self, dh, permuteOut, recvCounts, gateWeight, upWeight, saved, want_rows=True, want_weights=True,
                 dAtaOut=None, dGate=None, dUp=None, stream=None) -> GatedGrads:
        d, dtype, ws, device = self.desc, self.dtype, self.workspace, self.workspace.get_device()
        A, H1, N = d.A, d.H1, d.N
        _is(dh, "dh", dtype, (A, N), device)
        _is(permuteOut, "permuteOut", dtype, (A, H1), device)
        self._check_shared(recvCounts, gateWeight, upWeight, device)
        _is(saved, "saved", torch.float32, (2, A, N), device)
        rows = _out(dAtaOut, "dAtaOut", dtype, (A, H1), permuteOut, stream) if want_rows else None
        gate = _out(dGate, "dGate", dtype, (d.e, H1, N), gateWeight, stream) if want_weights else None
        up = _out(dUp, "dUp", dtype, (d.e, H1, N), upWeight, stream) if want_weights else None
        _enqueue("a2av_gated_backward", device, stream, ctypes.byref(d), dh.data_ptr(), permuteOut.data_ptr(),
                 recvCounts.data_ptr(), gateWeight.data_ptr(), upWeight.data_ptr(), saved.data_ptr(), _at(rows), _at(gate),
                 _at(up), ws.data_ptr(), ws.numel())
        return GatedGrads(rows, gate, up)


class GmmBackwardPlan:
    """Descriptor + workspace of the grouped product's gradients for one shape (a2av_gmm_backward)."""

    def __init__(self, W, e, A, H1, N1, dtype=torch.bfloat16, device=None):
        self.desc = make_desc(W, e, A, H1, N1, dtype=dtype)
        self.dtype = dtype
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.workspace = torch.empty(_size("a2av_gmm_backward_workspace_size", ctypes.byref(self.desc)),
                                     dtype=torch.uint8, device=self.device)

    def run(self, dY, permuteOut, recvCounts, gmmWeight, want_rows=True, want_weights=True, dAtaOut=None,
            dWeight=None, stream=None):
        """(dAtaOut [A, H1] rank-major, dWeight [e, H1, N1]); either may be left out (None)."""
        d, dtype, ws, device = self.desc, self.dtype, self.workspace, self.workspace.get_device()
        A, H1, N1 = d.A, d.H1, d.N1
        _is(dY, "dY", dtype, (A, N1), device)
        _is(permuteOut, "permuteOut", dtype, (A, H1), device)
        _is(recvCounts, "recvCounts", torch.int32, (d.W * d.e,), device)
        _is(gmmWeight, "gmmWeight", dtype, (d.e, H1, N1), device)
        rows = _out(dAtaOut, "dAtaOut", dtype, (A, H1), permuteOut, stream) if want_rows else None
        weights = _out(dWeight, "dWeight", dtype, (d.e, H1, N1), gmmWeight, stream) if want_weights else None
        _enqueue("a2av_gmm_backward", device, stream, ctypes.byref(d), dY.data_ptr(), permuteOut.data_ptr(),
                 recvCounts.data_ptr(), gmmWeight.data_ptr(), _at(rows), _at(weights), ws.data_ptr(), ws.numel())
        return rows, weights


# ---- the product of 8-bit rows with a float32 scale per 128 (include/a2av_gmm_g128.h)


class G128Plan:
    """Descriptor + workspace of the grouped product of codes with a float32 scale for each 128, for one shape: rows as
    a2av_rms_norm, a2av_layer_norm and a2av_glu_quant write them in mode "group128", weights [e, N1, H1] with a scale
    for 128 columns x 128 codes.  dtype: of the output.  The workspace serves one call at a time: calls of one plan on
    different streams have to be ordered by the caller."""

    def __init__(self, W, e, A, H1, N1, dtype=torch.bfloat16, qtype="e4m3fn", device=None):
        if dtype not in DTYPES:
            raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
        self.desc = G128Desc(W, e, A, H1, N1, DTYPES[dtype], _named(QTYPES, qtype, "qtype"))
        self.dtype = dtype
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.workspace = torch.empty(_size("a2av_gmm_g128_workspace_size", ctypes.byref(self.desc)), dtype=torch.uint8,
                                     device=self.device)

    def run(self, ataOut_q, ataOut_s, recvCounts, gmmWeight_q, gmmWeight_s, gmmY=None, stream=None):
        """gmmY [A, N1], expert-major, from ataOut_q uint8 [A, H1] and ataOut_s float32 [A, H1/128] (rank-major),
        gmmWeight_q uint8 [e, N1, H1] and gmmWeight_s float32 [e, ceil(N1/128), H1/128]."""
        d, ws, device = self.desc, self.workspace, self.workspace.get_device()
        A, H1, N1 = d.A, d.H1, d.N1
        _is(ataOut_q, "ataOut_q", torch.uint8, (A, H1), device)
        _is(ataOut_s, "ataOut_s", torch.float32, (A, H1 // 128), device)
        _is(recvCounts, "recvCounts", torch.int32, (d.W * d.e,), device)
        _is(gmmWeight_q, "gmmWeight_q", torch.uint8, (d.e, N1, H1), device)
        _is(gmmWeight_s, "gmmWeight_s", torch.float32, (d.e, -(-N1 // 128), H1 // 128), device)
        gmmY = _out(gmmY, "gmmY", self.dtype, (A, N1), ws, stream)
        _enqueue("a2av_gmm_g128_run", device, stream, ctypes.byref(d), ataOut_q.data_ptr(), ataOut_s.data_ptr(),
                 recvCounts.data_ptr(), gmmWeight_q.data_ptr(), gmmWeight_s.data_ptr(), gmmY.data_ptr(), ws.data_ptr(),
                 ws.numel())
        return gmmY


# ---- a whole expert layer for a few tokens (include/a2av_moe.h)


class MoeOut(NamedTuple):
    y: torch.Tensor        # [T, H]
    experts: torch.Tensor  # int32 [T, K], the largest score (+ bias) first
    weights: torch.Tensor  # float32 [T, K]


class MoePlan:
    """Descriptor + workspace of a whole expert layer for T tokens (up to 64): the router's choice of K of E experts, their
    gated blocks and down projections, and the weighted sum.  score: "softmax" or "sigmoid"; renormalise: the chosen scores
    are divided by their sum; scale: of the weights; router_dtype: dtype or float32.  The workspace serves one call at a
    time: calls of one plan on different streams have to be ordered by the caller."""

    def __init__(self, T, E, K, H, N, dtype=torch.bfloat16, act="silu", score="softmax", renormalise=True, scale=1.0,
                 router_dtype=None, device=None):
        if dtype not in DTYPES:
            raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
        self.router_dtype = dtype if router_dtype is None else router_dtype
        if self.router_dtype not in (dtype, torch.float32):
            raise TypeError(f"router_dtype must be {dtype} or float32, got {router_dtype}")
        self.desc = MoeDesc(T, E, K, H, N, DTYPES[dtype], 2 if self.router_dtype == torch.float32 else DTYPES[dtype],
                            _named(ACTS, act, "act"), _named(SCORES, score, "score"), int(bool(renormalise)), scale)
        self.dtype = dtype
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.workspace = torch.empty(_size("a2av_moe_workspace_size", ctypes.byref(self.desc)), dtype=torch.uint8,
                                     device=self.device)

    def run(self, x, router, gate, up, down, bias=None, residual=None, out: Optional[MoeOut] = None,
            stream=None) -> MoeOut:
        """x [T, H], router [E, H], gate and up [E, H, N], down [E, N, H], bias float32 [E] (added to the scores for the
        choice only), residual [T, H] (added to the result).  `out`: an earlier result, whose tensors are written again;
        its y may be x or the residual."""
        d, dtype, ws, device = self.desc, self.dtype, self.workspace, self.workspace.get_device()
        T, E, K, H, N = d.T, d.E, d.K, d.H, d.N
        _is(x, "x", dtype, (T, H), device)
        _is(router, "router", self.router_dtype, (E, H), device)
        _is(gate, "gate", dtype, (E, H, N), device)
        _is(up, "up", dtype, (E, H, N), device)
        _is(down, "down", dtype, (E, N, H), device)
        if bias is not None:
            _is(bias, "bias", torch.float32, (E,), device)
        if residual is not None:
            _is(residual, "residual", dtype, (T, H), device)
        y = _out(out.y if out else None, "y", dtype, (T, H), x, stream)
        experts = _out(out.experts if out else None, "experts", torch.int32, (T, K), ws, stream)
        weights = _out(out.weights if out else None, "weights", torch.float32, (T, K), ws, stream)
        _enqueue("a2av_moe_run", device, stream, ctypes.byref(d), x.data_ptr(), router.data_ptr(), _at(bias),
                 gate.data_ptr(), up.data_ptr(), down.data_ptr(), _at(residual), y.data_ptr(), experts.data_ptr(),
                 weights.data_ptr(), ws.data_ptr(), ws.numel())
        return MoeOut(y, experts, weights)
