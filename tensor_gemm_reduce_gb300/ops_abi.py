"""ctypes signatures of include/gemm_rs_ops.h and what its bindings share.

The operators live in the same library as gemm_rs.py's and report the same
status codes; a failure raises GemmRSError, a tensor of a wrong type, shape or
device raises TypeError or ValueError before the library is called.

Calls that a step makes go through a compiled entry (csrc/ops_binding.cpp):
checking a call's tensors here took 8 to 11 us, longer than the smallest
operators run.  What is called once (layouts, plans, packing) uses ctypes.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import re
from typing import Optional

import torch

from . import build as _build
from . import gemm_rs as _g

GemmRSError = _g.GemmRSError
WORLD = _g.WORLD
NORM_MAX_D = 16384

_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class gemm_rs_norm_desc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("D", ctypes.c_int64), ("gate_rows", ctypes.c_int64),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


# Every entry point declared in include/gemm_rs_ops.h.
SIGS = {
    "gemm_rs_norm_forward": [_P] * 10,
    "gemm_rs_norm_workspace": [_P, _P],
    "gemm_rs_norm_backward": [_P] * 16,
    "gemm_rs_act8_layout": [_L, _L, _P, _P, _P],
    "gemm_rs_act8_save": [_L, _L, _P, _P, _P, _P],
    "gemm_rs_act8_restore": [_L, _L, _P, _P, _P, _P],
    "gemm_rs_bwd_create": [_L, _L, _L, ctypes.c_uint64, _P, _P],
    "gemm_rs_bwd_run": [_P] * 9,
    "gemm_rs_bwd_status": [_P, _P],
    "gemm_rs_bwd_destroy": [_P],
    "gemm_rs_w4_bytes": [_L, _L, _I, _I, _P],
    "gemm_rs_w4_quantize": [_L, _L, _I, _P, _P, _P, _P],
    "gemm_rs_w4_pack": [_L, _L, _I, _P, _P, _P, _P, _P],
    "gemm_rs_w4_run": [_L, _L, _L, _I, _I, _P, _P, _P, _P],
}

_LIB: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The library with these entry points declared (built first if it is missing)."""
    global _LIB
    if _LIB is None:
        cdll = _g.load_library()
        for name, args in SIGS.items():
            fn = getattr(cdll, name)
            fn.restype, fn.argtypes = _I, args
        _LIB = cdll
    return _LIB


_OPS = None


def ops():
    """The compiled entry of the operators (built first if there is none of these sources)."""
    global _OPS
    if _OPS is None:
        lib()
        path = _build.build_binding()
        loader = importlib.machinery.ExtensionFileLoader("_ops", path)
        spec = importlib.util.spec_from_file_location("_ops", path, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _OPS = module
    return _OPS


def header_symbols():
    """Names of the functions declared in include/gemm_rs_ops.h."""
    text = open(os.path.join(_build.ROOT, "include", "gemm_rs_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gemm_rs_[a-z0-9_]+)\s*\(", text)))


def check(rc: int, what: str) -> None:
    if rc != _g.GEMM_RS_OK:
        raise GemmRSError(rc, what)


_AS_IT_IS = contextlib.nullcontext()


def allocating_for(stream):
    """Context for what a call allocates when it runs on `stream`: the memory then belongs
    to that stream.  From the current stream's memory a call could be given a block that
    this stream's earlier work still reads, and a temporary that the call drops could go to
    the current stream's next allocation before `stream` has used it."""
    return _AS_IT_IS if stream is None else torch.cuda.stream(stream)


def pointer(t, shape, dtype, name: str, device=None) -> int:
    """Address of a contiguous CUDA tensor of this shape and dtype (on `device`)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.data_ptr()


def stream_handle(stream, device) -> int:
    """The stream's handle, or the current stream's; `device` must be the current device."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream
