"""The row-parallel layer's input kept in 8 bits between its forward and its
backward pass, and the backward pass (binding of gemm_rs_act8_* and
gemm_rs_bwd_* in include/gemm_rs_ops.h).

    ck = act8.save(A)                      A [8][M][K/8] bf16 -> 1.03 bytes an element
    plan = act8.BackwardPlan(M, N, K)
    plan.run(dY, W, ck, dA, dW, plan.new_workspace())

32 consecutive elements of a row share a power of two, the least that holds
the largest of them in 7 bits and a sign; a restored value is exact in bf16.
A group with an infinity or a NaN is restored as NaN.

Calls run on `stream`, or the current one, and what they allocate belongs to it.
"""
from __future__ import annotations

import ctypes

import torch

from . import ops_abi as _a

GROUP = 32
_BF16, _U8 = torch.bfloat16, torch.uint8


class Checkpoint:
    """Storage of one checkpoint of A [8][M][K/8] (uninitialised): `codes` and
    `scales` are private to the library, move them as they are."""

    def __init__(self, M: int, K: int, device=None):
        self.M, self.K = int(M), int(K)
        self.shape = torch.Size((_a.WORLD, self.M, self.K // _a.WORLD))
        pitch, cb, sb = ctypes.c_int64(), ctypes.c_size_t(), ctypes.c_size_t()
        _a.check(_a.lib().gemm_rs_act8_layout(self.M, self.K, ctypes.byref(pitch), ctypes.byref(cb),
                                              ctypes.byref(sb)), "gemm_rs_act8_layout")
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.codes = torch.empty(_a.WORLD, self.M, pitch.value, dtype=_U8, device=device)
        self.scales = torch.empty(_a.WORLD, self.M, pitch.value // GROUP, dtype=_U8, device=device)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def save(A, out: Checkpoint = None, stream=None) -> Checkpoint:
    """A checkpoint of A [8][M][K/8]; `out` is written when given."""
    if A.dim() != 3 or A.shape[0] != _a.WORLD:
        raise ValueError(f"A must have shape [{_a.WORLD}][M][K/{_a.WORLD}], got {tuple(A.shape)}")
    if out is None:
        with _a.allocating_for(stream):
            out = Checkpoint(A.shape[1], A.shape[2] * _a.WORLD, A.device)
    elif out.shape != A.shape:
        raise ValueError(f"the checkpoint holds {tuple(out.shape)}, A is {tuple(A.shape)}")
    rc = _a.ops().act8(A, out.codes, out.scales, False, None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_act8_save")
    return out


def restore(ck: Checkpoint, out=None, stream=None):
    """The bf16 values [8][M][K/8] that a checkpoint stands for."""
    if out is None:
        with _a.allocating_for(stream):
            out = torch.empty(ck.shape, dtype=_BF16, device=ck.codes.device)
    elif out.shape != ck.shape:
        raise ValueError(f"the checkpoint holds {tuple(ck.shape)}, out is {tuple(out.shape)}")
    rc = _a.ops().act8(out, ck.codes, ck.scales, True, None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_act8_restore")
    return out


class BackwardPlan:
    """Backward pass of out = sum_r A_r W_r for one (M, N, K) on the current device:
    dA[r] = dY W[r]^T and dW[r] = A[r]^T dY."""

    def __init__(self, M: int, N: int, K: int, *, timeout_ns: int = 0):
        self.M, self.N, self.K = int(M), int(N), int(K)
        h, ws = ctypes.c_void_p(), ctypes.c_size_t()
        _a.check(_a.lib().gemm_rs_bwd_create(self.M, self.N, self.K, timeout_ns, ctypes.byref(h),
                                             ctypes.byref(ws)), "gemm_rs_bwd_create")
        self._h, self.workspace_bytes, self._workspace = h.value, ws.value, None
        Kr = self.K // _a.WORLD
        self.a_shape = torch.Size((_a.WORLD, self.M, Kr))
        self.w_shape = torch.Size((_a.WORLD, Kr, self.N))

    def new_workspace(self, device=None):
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        return torch.empty(self.workspace_bytes, dtype=_U8, device=device)

    def run(self, dY, W, checkpoint, dA, dW, workspace, stream=None) -> None:
        """Enqueue one pass.  dA may be None (W is then not read), and so may dW (the
        checkpoint is then not read)."""
        codes = scales = None
        if dW is not None:
            if checkpoint.shape != self.a_shape:
                raise ValueError(f"the checkpoint holds {tuple(checkpoint.shape)}, the plan {tuple(self.a_shape)}")
            codes, scales = checkpoint.codes, checkpoint.scales
        rc = _a.ops().backward(self._h, self.M, self.N, self.K, self.workspace_bytes, dY, W, codes, scales, dA, dW,
                               workspace, None if stream is None else stream.cuda_stream)
        if rc:
            _a.check(rc, "gemm_rs_bwd_run")
        self._workspace = workspace  # status() reads it

    def status(self, stream=None) -> int:
        """Synchronise the stream and report the device-side status of the last run, whose
        workspace the plan keeps for this until its next run or close()."""
        s = stream if stream is not None else torch.cuda.current_stream()
        return _a.lib().gemm_rs_bwd_status(self._h, s.cuda_stream)

    def close(self):
        if getattr(self, "_h", None):
            _a.lib().gemm_rs_bwd_destroy(self._h)
            self._h = self._workspace = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
