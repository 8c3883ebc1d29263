"""The row-parallel layer in 8-bit floating point (e4m3) with a scale for each
block of 128, forward and backward (binding of gemm_rs_fp8_* in
include/gemm_rs_ops.h).

    weight = fp8.quantize(W)                         W [8][K/8][N] bf16, 128 x 128 blocks
    out = fp8.forward(A, weight, checkpoint=ck)      out = sum_r A_r W_r, A [8][M][K/8]
    dA, dW = fp8.backward(dY, weight, ck)            dA_r = dY W_r^T, dW_r = A_r^T dY

A is quantised in 1 x 128 blocks along K/8, dY along N for dA; for dW both are
quantised in blocks of 128 tokens, A's by forward() into `ck`.  A block's scale is
its largest magnitude / 448 in fp32; products are summed in fp32 and rounded to bf16
once.  A block with an infinity or a NaN makes NaN of the outputs that it takes part in.

A weight of quantize(W, scales=torch.float8_e8m0fnu) has powers of two instead, the
least whose 448-fold holds the block, and so have the inputs and gradients that are
multiplied by it.  The tensor cores apply these by themselves: products of many tokens
take 0.6 to 0.8 of the time, and are less accurate (inputs with one entry in 20 eight times
as large are rounded by 2.7% of their norm, with fp32 by 2.1%).

Weights of several experts, W [E][8][K/8][N], are quantised alike; moe.py
multiplies by them.

Calls run on `stream`, or the current one, and what they allocate belongs to it.
"""
from __future__ import annotations

import ctypes

import torch

from . import ops_abi as _a

BLOCK = 128
_BF16, _F32, _U8, _E4M3, _E8M0 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.float8_e8m0fnu
_default_scales = _F32


def default_scales() -> torch.dtype:
    """The type of the scales of weights that are made without naming one."""
    return _default_scales


def set_default_scales(dtype: torch.dtype) -> None:
    """torch.float32 (the default), or torch.float8_e8m0fnu: powers of two."""
    global _default_scales
    _default_scales = _scale_type(dtype)


def _scale_type(dtype) -> torch.dtype:
    if dtype is None:
        return _default_scales
    if dtype not in (_F32, _E8M0):
        raise ValueError(f"scales must be {_F32} or {_E8M0}, got {dtype}")
    return dtype


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


class Weight:
    """Codes and scales of one weight (experts=None) or of several experts', uninitialised.

    storage: [E][8][ceil(N/128)][K/8][128] torch.float8_e4m3fn, 128 columns of W at a time, zero
    behind the last; scales: [E][8][ceil(K/8/128)][ceil(N/128)] fp32 or torch.float8_e8m0fnu
    (`scales`; None: default_scales()); both without [E] for one weight.  Fill them with quantize(),
    or with load()."""

    def __init__(self, N: int, K: int, experts=None, device=None, scales: torch.dtype = None):
        self.N, self.K, self.experts = int(N), int(K), None if experts is None else int(experts)
        E = 1 if experts is None else self.experts
        scales = _scale_type(scales)
        cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
        _a.check(_a.lib().gemm_rs_fp8_weight_bytes(E, self.N, self.K, ctypes.byref(cb), ctypes.byref(sb)),
                 "gemm_rs_fp8_weight_bytes")
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        Kr = self.K // _a.WORLD
        lead = (_a.WORLD,) if experts is None else (E, _a.WORLD)
        self.shape = torch.Size((*lead, Kr, self.N))
        self.storage = torch.empty(*lead, _blocks(self.N), Kr, BLOCK, dtype=_E4M3, device=device)
        self.scales = torch.empty(*lead, _blocks(Kr), _blocks(self.N), dtype=scales, device=device)

    def load(self, codes, scales) -> "Weight":
        """Take codes of this weight's shape (torch.float8_e4m3fn) and scales of its type, made elsewhere;
        a weight with fp32 scales takes powers of two as well."""
        if codes.dtype is not _E4M3 or scales.dtype not in (self.scales.dtype, _E8M0):
            raise TypeError(f"codes and scales must be {_E4M3} and {self.scales.dtype}, got {codes.dtype} and {scales.dtype}")
        if codes.shape != self.shape or scales.shape != self.scales.shape:
            raise ValueError(f"codes and scales must have shapes {tuple(self.shape)} and {tuple(self.scales.shape)}, "
                             f"got {tuple(codes.shape)} and {tuple(scales.shape)}")
        whole = torch.nn.functional.pad(codes.view(_U8), (0, -self.N % BLOCK))
        self.storage.view(_U8).copy_(whole.unflatten(-1, (-1, BLOCK)).transpose(-3, -2))
        if scales.dtype is self.scales.dtype:
            self.scales.view(_U8).copy_(scales.view(_U8))
        else:
            self.scales.copy_(scales.float())
        return self

    @property
    def codes(self):
        """A copy of the codes in the weight's own shape."""
        return self.storage.view(_U8).transpose(-3, -2).flatten(-2)[..., :self.N].contiguous().view(_E4M3)


def quantize(W, out: Weight = None, stream=None, scales: torch.dtype = None) -> Weight:
    """The codes and scales (torch.float32 or torch.float8_e8m0fnu; None: default_scales(), or out's) of
    W [8][K/8][N] or [E][8][K/8][N] bf16; `out` is written when given."""
    if W.dim() not in (3, 4) or W.shape[-3] != _a.WORLD:
        raise ValueError(f"W must have shape [{_a.WORLD}][K/{_a.WORLD}][N] or [E][{_a.WORLD}][K/{_a.WORLD}][N], "
                         f"got {tuple(W.shape)}")
    if out is None:
        with _a.allocating_for(stream):
            out = Weight(W.shape[-1], W.shape[-2] * _a.WORLD, None if W.dim() == 3 else W.shape[0], W.device, scales)
    elif out.shape != W.shape:
        raise ValueError(f"the weight has shape {tuple(out.shape)}, W is {tuple(W.shape)}")
    elif scales not in (None, out.scales.dtype):
        raise ValueError(f"the weight's scales are {out.scales.dtype}, not {scales}")
    rc = _a.ops().fp8_quantize(W, out.storage, out.scales, None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_fp8_quantize")
    return out


class Checkpoint:
    """What backward() needs of A [8][M][K/8] (uninitialised): its codes in blocks of 128
    tokens.  `codes` and `scales` are private to the library, move them as they are; scale_type is
    that of the weight of the forward() that wrote them, and backward()'s has to be the same."""

    def __init__(self, M: int, K: int, device=None):
        self.M, self.K = int(M), int(K)
        cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
        _a.check(_a.lib().gemm_rs_fp8_checkpoint_bytes(self.M, self.K, ctypes.byref(cb), ctypes.byref(sb)),
                 "gemm_rs_fp8_checkpoint_bytes")
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.codes = torch.empty(cb.value, dtype=_U8, device=device)
        self.scales = torch.empty(sb.value, dtype=_U8, device=device)
        self.scale_type = None

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def check_scale_type(checkpoint, weight: Weight):
    if checkpoint is not None and checkpoint.scale_type not in (None, weight.scales.dtype):
        raise ValueError(f"the checkpoint was written with a weight whose scales are {checkpoint.scale_type}, "
                         f"this one's are {weight.scales.dtype}")


def _one(weight: Weight):
    if weight.experts is not None:
        raise ValueError("the weight is of several experts: see moe.forward and moe.backward")


def workspace_bytes(M: int, weight: Weight) -> int:
    n = ctypes.c_size_t()
    _a.check(_a.lib().gemm_rs_fp8_workspace(M, weight.N, weight.K, ctypes.byref(n)), "gemm_rs_fp8_workspace")
    return n.value


def new_workspace(M: int, weight: Weight):
    """Workspace of forward() and backward() for M tokens (uninitialised)."""
    return torch.empty(workspace_bytes(M, weight), dtype=_U8, device=weight.scales.device)


def new_gradients(M: int, weight: Weight):
    """(dA, dW) for backward(out=...)."""
    device = weight.scales.device
    return (torch.empty(_a.WORLD, M, weight.K // _a.WORLD, dtype=_BF16, device=device),
            torch.empty(weight.shape, dtype=_BF16, device=device))


def forward(A, weight: Weight, checkpoint: Checkpoint = None, out=None, workspace=None, stream=None):
    """out [M][N] = sum_r A_r W_r for A [8][M][K/8]; `checkpoint` is written when given."""
    _one(weight)
    if A.dim() != 3:
        raise ValueError(f"A must have shape [{_a.WORLD}][M][K/{_a.WORLD}], got {tuple(A.shape)}")
    M = A.shape[1]
    if checkpoint is not None and (checkpoint.M, checkpoint.K) != (M, weight.K):
        raise ValueError(f"the checkpoint is for M = {checkpoint.M}, K = {checkpoint.K}, A is {tuple(A.shape)}")
    if out is None or workspace is None:
        with _a.allocating_for(stream):
            out = torch.empty(M, weight.N, dtype=_BF16, device=A.device) if out is None else out
            workspace = new_workspace(M, weight) if workspace is None else workspace
    codes, scales = (None, None) if checkpoint is None else (checkpoint.codes, checkpoint.scales)
    rc = _a.ops().fp8_forward(A, M, weight.N, weight.K, weight.storage, weight.scales, codes, scales, out, workspace,
                              None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_fp8_forward")
    if checkpoint is not None:
        checkpoint.scale_type = weight.scales.dtype
    return out


def backward(dY, weight: Weight, checkpoint: Checkpoint, out=None, workspace=None, stream=None):
    """(dA, dW) for dY [M][N], the gradient of forward()'s result.  `out` takes the tensors
    of new_gradients(); where one of them is None that gradient is not computed, and without dW
    `checkpoint` may be None."""
    _one(weight)
    if dY.dim() != 2:
        raise ValueError(f"dY must have shape [M][{weight.N}], got {tuple(dY.shape)}")
    M = dY.shape[0]
    if out is None or workspace is None:
        with _a.allocating_for(stream):
            out = new_gradients(M, weight) if out is None else out
            workspace = new_workspace(M, weight) if workspace is None else workspace
    dA, dW = out
    codes = scales = None
    if dW is not None:
        if checkpoint is None:
            raise ValueError("dW needs the checkpoint")
        if (checkpoint.M, checkpoint.K) != (M, weight.K):
            raise ValueError(f"the checkpoint is for M = {checkpoint.M}, K = {checkpoint.K}, dY is {tuple(dY.shape)}")
        check_scale_type(checkpoint, weight)
        codes, scales = checkpoint.codes, checkpoint.scales
    rc = _a.ops().fp8_backward(dY, M, weight.N, weight.K, weight.storage, weight.scales, codes, scales, dA, dW,
                               workspace, None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_fp8_backward")
    return dA, dW


def status(workspace, stream=None) -> int:
    """Synchronise the stream and report the device-side status of the last call of forward()
    or backward() (here or in moe.py) that used this workspace."""
    if workspace.dtype is not _U8 or workspace.numel() < 4:
        raise ValueError("not a workspace of these calls")
    return _a.lib().gemm_rs_fp8_status(_a.pointer(workspace, workspace.shape, _U8, "workspace"),
                                       _a.stream_handle(stream, workspace.device))
