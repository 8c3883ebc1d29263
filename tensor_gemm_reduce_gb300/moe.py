"""Routing to experts, and the experts' row-parallel layer in 8-bit floating
point, forward and backward (binding of gemm_rs_moe_* in include/gemm_rs_ops.h).

    routing = moe.route(logits, 2)                       ids, weights, rows of [T][k], offsets [E+1]
    weight = fp8.quantize(W)                             W [E][8][K/8][N] bf16
    out = moe.forward(A, weight, routing, checkpoint=ck) out[t] = sum_j weights[t][j] A[row] W[expert]
    dA, dW, dweights = moe.backward(dout, weight, routing, ck)
    dlogits = moe.route_backward(dweights, logits, routing)

A [8][T*k][K/8] bf16 holds the input of each token-expert pair at its place in the
order of the experts: row rows[t][j] belongs to token t and its j-th expert, and
x[routing.pairs // k] brings the tokens' rows into that order.  Blocks, scales and
rounding are fp8.py's; weights and sums over a token's experts are fp32.

Calls run on `stream`, or the current one, and what they allocate belongs to it.
"""
from __future__ import annotations

import ctypes

import torch

from . import fp8 as _f
from . import ops_abi as _a

MAX_TOP_K = 16
MAX_EXPERTS = 256
_SCORES = {"softmax": 0, "sigmoid": 1}
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Routing:
    """T tokens' k experts out of E (uninitialised): ids and weights [T][k], descending by
    choice; rows [T][k], each pair's place in the order of the experts (-1 without an expert);
    pairs [T*k], the pair t*k + j at each place, and behind the last one with an expert 0 or what an
    earlier call left there, so that every place is an index; offsets [E+1], each expert's first place
    and, last, the number of pairs with an expert."""

    def __init__(self, T: int, k: int, E: int, device=None):
        self.T, self.k, self.E = int(T), int(k), int(E)
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.ids, self.rows = (torch.empty(self.T, self.k, dtype=_I32, device=device) for _ in range(2))
        self.weights = torch.empty(self.T, self.k, dtype=_F32, device=device)
        # places behind the last pair with an expert are never written: they hold a pair that there is
        self.pairs = torch.zeros(self.T * self.k, dtype=_I32, device=device)
        self.offsets = torch.empty(self.E + 1, dtype=_I32, device=device)
        self.options = None  # how route() chose: (score, groups, top_groups, renormalize, scale)


def route(logits, k: int, bias=None, score: str = "softmax", groups: int = 1, top_groups: int = None,
          renormalize: bool = True, scale: float = 1.0, mask=None, out: Routing = None, stream=None) -> Routing:
    """The k experts of each token, from logits [T][E] (fp32 or bf16).

    Scores are a softmax over the experts or each one's sigmoid; the choice is by score + bias
    (bias [E] fp32), within the top_groups of `groups` groups of consecutive experts whose two
    best choices have the largest sums; equal choices go to the lower index.  Weights are the
    scores, over the sum of the chosen ones if `renormalize`, times `scale`.  Tokens where mask
    [T] (bool) is False get no expert: ids and rows -1, weights 0."""
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if logits.dim() != 2:
        raise ValueError(f"logits must have shape [T][E], got {tuple(logits.shape)}")
    T, E = logits.shape
    if out is None:
        if not 1 <= k <= MAX_TOP_K:
            raise ValueError(f"k must be from 1 to {MAX_TOP_K}, got {k}")
        with _a.allocating_for(stream):
            out = Routing(T, k, E, logits.device)
    elif (out.T, out.k, out.E) != (T, k, E):
        raise ValueError(f"the routing is of T, k, E = {out.T, out.k, out.E}, not {T, k, E}")
    options = (_SCORES[score], groups, groups if top_groups is None else top_groups, renormalize, scale)
    rc = _a.ops().moe_route(logits, bias, mask, k, *options, out.ids, out.weights, out.rows, out.pairs, out.offsets,
                            None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_moe_route")
    out.options = options
    return out


def route_backward(dweights, logits, routing: Routing, out=None, stream=None):
    """dlogits [T][E], of the logits' type, for dweights [T][k] fp32, the gradient of route()'s
    weights.  The choice of experts and the bias have no gradient."""
    if routing.options is None:
        raise ValueError("the routing is not of route()")
    if out is None:
        with _a.allocating_for(stream):
            out = torch.empty_like(logits)
    rc = _a.ops().moe_route_backward(dweights, logits, routing.ids, routing.k, *routing.options, out,
                                     None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_moe_route_backward")
    return out


def arrange(ids, weights, E: int, out: Routing = None, stream=None) -> Routing:
    """A Routing of ids [T][k] int32 and weights [T][k] fp32 that were chosen elsewhere (the tensors
    themselves, not copies: route() into the same Routing writes to them); an id outside 0 .. E-1 is
    no expert."""
    if ids.dim() != 2:
        raise ValueError(f"ids must have shape [T][k], got {tuple(ids.shape)}")
    _a.pointer(weights, ids.shape, _F32, "weights", ids.device)
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"E must be from 1 to {MAX_EXPERTS}, got {E}")
    if out is None:
        with _a.allocating_for(stream):
            out = Routing(*ids.shape, E, ids.device)
    elif (out.T, out.k, out.E) != (*ids.shape, E):
        raise ValueError(f"the routing is of T, k, E = {out.T, out.k, out.E}, not {(*ids.shape, E)}")
    rc = _a.ops().moe_arrange(ids, E, out.rows, out.pairs, out.offsets, None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_moe_arrange")
    out.ids, out.weights, out.options = ids, weights, None
    return out


def _desc(routing: Routing, weight: _f.Weight):
    if weight.experts != routing.E:
        raise ValueError(f"the weight has {weight.experts or 'no'} experts, the routing {routing.E}")
    return _a.gemm_rs_moe_desc(routing.T, routing.E, routing.k, weight.N, weight.K)


class Checkpoint:
    """What backward() needs of forward() (uninitialised): A's codes in blocks of 128 of an
    expert's rows, private to the library, and y [T*k][N] fp32, each pair's product."""

    def __init__(self, routing: Routing, weight: _f.Weight):
        d = _desc(routing, weight)
        cb, sb, yb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        _a.check(_a.lib().gemm_rs_moe_checkpoint_bytes(ctypes.byref(d), ctypes.byref(cb), ctypes.byref(sb),
                                                       ctypes.byref(yb)), "gemm_rs_moe_checkpoint_bytes")
        self.key = (d.T, d.E, d.top_k, d.N, d.K)
        device = weight.scales.device
        self.codes = torch.empty(cb.value, dtype=_U8, device=device)
        self.scales = torch.empty(sb.value, dtype=_U8, device=device)
        self.y = torch.empty(d.T * d.top_k, d.N, dtype=_F32, device=device)
        self.scale_type = None  # as fp8.Checkpoint's


def workspace_bytes(routing: Routing, weight: _f.Weight) -> int:
    n = ctypes.c_size_t()
    _a.check(_a.lib().gemm_rs_moe_workspace(ctypes.byref(_desc(routing, weight)), ctypes.byref(n)),
             "gemm_rs_moe_workspace")
    return n.value


def new_workspace(routing: Routing, weight: _f.Weight):
    """Workspace of forward() and backward() (uninitialised)."""
    return torch.empty(workspace_bytes(routing, weight), dtype=_U8, device=weight.scales.device)


def new_gradients(routing: Routing, weight: _f.Weight):
    """(dA, dW, dweights) for backward(out=...)."""
    device = weight.scales.device
    return (torch.empty(_a.WORLD, routing.T * routing.k, weight.K // _a.WORLD, dtype=_BF16, device=device),
            torch.empty(weight.shape, dtype=_BF16, device=device), torch.empty(routing.T, routing.k, dtype=_F32, device=device))


def _check(routing: Routing, weight: _f.Weight, checkpoint):
    d = _desc(routing, weight)
    key = (d.T, d.E, d.top_k, d.N, d.K)
    if checkpoint is not None and checkpoint.key != key:
        raise ValueError(f"the checkpoint is for T, E, k, N, K = {checkpoint.key}, not {key}")
    return key


def forward(A, weight: _f.Weight, routing: Routing, checkpoint: Checkpoint = None, out=None, workspace=None, stream=None):
    """out [T][N], the weighted sum of each token's experts' products; `checkpoint` is written when
    given.  Rows of A behind the last pair with an expert are not read."""
    key = _check(routing, weight, checkpoint)
    if out is None or workspace is None:
        with _a.allocating_for(stream):
            out = torch.empty(routing.T, weight.N, dtype=_BF16, device=A.device) if out is None else out
            workspace = new_workspace(routing, weight) if workspace is None else workspace
    kept = (None, None, None) if checkpoint is None else (checkpoint.codes, checkpoint.scales, checkpoint.y)
    rc = _a.ops().moe_forward(A, *key, weight.storage, weight.scales, routing.weights, routing.rows, routing.offsets,
                              *kept, out, workspace, None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_moe_forward")
    if checkpoint is not None:
        checkpoint.scale_type = weight.scales.dtype
    return out


def backward(dout, weight: _f.Weight, routing: Routing, checkpoint: Checkpoint, out=None, workspace=None, stream=None):
    """(dA, dW, dweights) for dout [T][N], the gradient of forward()'s result.  `out` takes the
    tensors of new_gradients(); where one of them is None that gradient is not computed, and with
    dA alone `checkpoint` may be None.  Rows of dA behind the last pair with an expert are left as they were."""
    if out is None or workspace is None:
        with _a.allocating_for(stream):
            out = new_gradients(routing, weight) if out is None else out
            workspace = new_workspace(routing, weight) if workspace is None else workspace
    dA, dW, dweights = out
    if checkpoint is None and (dW is not None or dweights is not None):
        raise ValueError("dW and dweights need the checkpoint")
    key = _check(routing, weight, checkpoint)
    _f.check_scale_type(checkpoint, weight)
    kept = (None, None, None) if checkpoint is None else (checkpoint.codes, checkpoint.scales, checkpoint.y)
    rc = _a.ops().moe_backward(dout, *key, weight.storage, weight.scales, routing.weights, routing.rows, routing.pairs,
                               routing.offsets, *kept, dA, dW, dweights, workspace,
                               None if stream is None else stream.cuda_stream)
    if rc:
        _a.check(rc, "gemm_rs_moe_backward")
    return dA, dW, dweights
