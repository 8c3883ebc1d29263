"""The norms after and before a transformer block, fused with the block's gate
and residual scale (binding of gemm_rs_norm_* in include/gemm_rs_ops.h).

    u = y / rms(y) * w_post            norm after the block, y its output
    r = x + scale * gate * u           gate and residual scale
    h = r / rms(r) * w_pre             norm before the next block

x, y, r, h: [M][D] bf16; w_post, w_pre: [D] bf16; gate: [G][D] bf16 or None,
its row i serving rows [i*M/G, (i+1)*M/G); rms(v) = sqrt(mean(v^2) + eps).
D is a multiple of 8, at most 16384.  Arithmetic is fp32, rounded once.

Calls run on `stream`, or the current one, and what they allocate belongs to it.
"""
from __future__ import annotations

import ctypes

import torch

from . import ops_abi as _a

_BF16, _F32 = torch.bfloat16, torch.float32


def _desc(x, gate, scale, eps):
    if x.dim() != 2:
        raise ValueError(f"x must have shape [M][D], got {tuple(x.shape)}")
    M, D = x.shape
    if gate is None:
        rows = 0
    elif gate.dim() != 2 or gate.shape[1] != D or gate.shape[0] < 1 or M % gate.shape[0]:
        raise ValueError(f"gate must have shape [G][{D}] with G a divisor of {M}, got {tuple(gate.shape)}")
    else:
        rows = gate.shape[0]
    return _a.gemm_rs_norm_desc(M, D, rows, scale, eps)


def new_outputs(x):
    """(r, h, stats) for forward(out=...): stats holds the rows' 1/rms(y) and 1/rms(r), [2][M] fp32."""
    return torch.empty_like(x), torch.empty_like(x), torch.empty(2, x.shape[0], dtype=_F32, device=x.device)


def new_gradients(x, gate=None):
    """(dx, dy, dw_post, dw_pre, dgate) for backward(out=...)."""
    w = torch.empty(2, x.shape[1], dtype=_BF16, device=x.device)
    return (torch.empty_like(x), torch.empty_like(x), w[0], w[1],
            None if gate is None else torch.empty_like(gate))


def workspace_bytes(x, gate=None) -> int:
    n = ctypes.c_size_t()
    _a.check(_a.lib().gemm_rs_norm_workspace(ctypes.byref(_desc(x, gate, 1.0, 0.0)), ctypes.byref(n)),
             "gemm_rs_norm_workspace")
    return n.value


def new_workspace(x, gate=None):
    """Workspace of backward() for tensors of these shapes (uninitialised)."""
    return torch.empty(workspace_bytes(x, gate), dtype=torch.uint8, device=x.device)


def forward(x, y, w_post, w_pre, gate=None, scale: float = 1.0, eps: float = 1e-6, out=None, stream=None):
    """Returns (r, h, stats); `out` takes the tensors of new_outputs()."""
    if out is None:
        with _a.allocating_for(stream):
            out = new_outputs(x)
    r, h, stats = out
    rc = _a.ops().norm_forward(x, y, w_post, w_pre, gate, scale, eps, r, h, stats,
                               None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_norm_forward")
    return r, h, stats


def backward(dr, dh, x, y, w_post, w_pre, stats, gate=None, scale: float = 1.0, out=None, workspace=None,
             stream=None):
    """Gradients (dx, dy, dw_post, dw_pre, dgate) for dr and dh, the gradients of
    forward()'s r and h; stats as forward() returned them; dgate is None without
    a gate.  `out` takes the tensors of new_gradients()."""
    if out is None or workspace is None:
        with _a.allocating_for(stream):
            out = new_gradients(x, gate) if out is None else out
            workspace = new_workspace(x, gate) if workspace is None else workspace
    dx, dy, dw_post, dw_pre, dgate = out
    rc = _a.ops().norm_backward(dr, dh, x, y, w_post, w_pre, gate, stats, scale, dx, dy, dw_post, dw_pre, dgate,
                                workspace, None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_norm_backward")
    return dx, dy, dw_post, dw_pre, dgate
