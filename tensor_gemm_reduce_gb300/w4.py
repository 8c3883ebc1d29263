"""The row-parallel layer for 1 to 32 tokens with 4-bit weights and group
scales (binding of gemm_rs_w4_* in include/gemm_rs_ops.h).

    weight = w4.pack(codes, scales, zeros, group=128)     once
    out = w4.matvec(x, weight)

    out[m][n] = sum_r sum_k x[r][m][k] (codes[r][k][n] - zeros[r][k//group][n]) scales[r][k//group][n]

x [8][M][K/8] bf16, codes [8][K/8][N] uint8 (0..15), scales and zeros
[8][ceil(K/8/group)][N] bf16 and uint8; without zeros 8 is subtracted.
quantize() makes symmetric codes of a bf16 weight.

Calls run on `stream`, or the current one, and what they allocate belongs to it.
"""
from __future__ import annotations

import ctypes

import torch

from . import ops_abi as _a

MAX_TOKENS = 32
_BF16, _U8 = torch.bfloat16, torch.uint8


class Weight:
    """Packed weights of one layer: `data` is private to the library."""

    def __init__(self, N: int, K: int, group: int, has_zeros: bool, device=None):
        self.N, self.K, self.group, self.has_zeros = int(N), int(K), int(group), bool(has_zeros)
        n = ctypes.c_size_t()
        _a.check(_a.lib().gemm_rs_w4_bytes(self.N, self.K, self.group, self.has_zeros, ctypes.byref(n)),
                 "gemm_rs_w4_bytes")
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.data = torch.empty(n.value, dtype=_U8, device=device)


def _groups(Kr: int, group: int) -> int:
    return -(-Kr // group) if group > 0 else 0


def quantize(W, group: int = 128, stream=None):
    """(codes, scales) of W [8][K/8][N] bf16: scale = bf16(max |w| / 7) over a group,
    code = 8 + round(w / scale)."""
    if W.dim() != 3 or W.shape[0] != _a.WORLD:
        raise ValueError(f"W must have shape [{_a.WORLD}][K/{_a.WORLD}][N], got {tuple(W.shape)}")
    _, Kr, N = W.shape
    w = _a.pointer(W, W.shape, _BF16, "W")
    with _a.allocating_for(stream):
        codes = torch.empty(W.shape, dtype=_U8, device=W.device)
        scales = torch.empty(_a.WORLD, _groups(Kr, group), N, dtype=_BF16, device=W.device)
    _a.check(_a.lib().gemm_rs_w4_quantize(N, Kr * _a.WORLD, group, w, codes.data_ptr(), scales.data_ptr(),
                                          _a.stream_handle(stream, W.device)), "gemm_rs_w4_quantize")
    return codes, scales


def pack(codes, scales, zeros=None, group: int = 128, stream=None) -> Weight:
    """Lay the weights out for matvec(), once."""
    if codes.dim() != 3 or codes.shape[0] != _a.WORLD:
        raise ValueError(f"codes must have shape [{_a.WORLD}][K/{_a.WORLD}][N], got {tuple(codes.shape)}")
    _, Kr, N = codes.shape
    per_group = torch.Size((_a.WORLD, _groups(Kr, group), N))
    c = _a.pointer(codes, codes.shape, _U8, "codes")
    s = _a.pointer(scales, per_group, _BF16, "scales", codes.device)
    z = None if zeros is None else _a.pointer(zeros, per_group, _U8, "zeros", codes.device)
    with _a.allocating_for(stream):
        weight = Weight(N, Kr * _a.WORLD, group, zeros is not None, codes.device)
    _a.check(_a.lib().gemm_rs_w4_pack(N, weight.K, group, c, s, z, weight.data.data_ptr(),
                                      _a.stream_handle(stream, codes.device)), "gemm_rs_w4_pack")
    return weight


def new_workspace(weight: Weight):
    """A placeholder for matvec()'s `workspace`: an empty tensor.  The sums meet in the SMs'
    shared memory; the two are there so that callers can treat this layer like the library's
    others."""
    return torch.empty(0, dtype=_U8, device=weight.data.device)


def matvec(x, weight: Weight, out=None, workspace=None, stream=None):
    """out [M][N] = the layer's output for x [8][M][K/8], M at most 32.  `workspace` is a
    placeholder: it is not used."""
    if out is None:
        if x.dim() != 3:
            raise ValueError(f"x must have shape [{_a.WORLD}][M][K/{_a.WORLD}], got {tuple(x.shape)}")
        with _a.allocating_for(stream):
            out = torch.empty(x.shape[1], weight.N, dtype=_BF16, device=x.device)
    rc = _a.ops().w4_matvec(x, weight.N, weight.K, weight.group, weight.has_zeros, weight.data, out,
                            None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_w4_run")
    return out
