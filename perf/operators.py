"""The operators around the row-parallel linear layer, as they are measured.

block_norm: the norms after and before a block with its gate and residual
scale, forward and backward; act8: the layer's input kept in 8 bits for
training, and the layer's backward pass from it; w4: the layer for single
tokens with 4-bit weights and group scales.  Shapes: M tokens, N (or D)
output columns, K inner dimension over 8 virtual ranks.
"""
import math

import torch

own = False

WORLD = 8
GROUP8 = 32  # elements that share a scale in an 8-bit checkpoint
EPS = 1e-6
SCALE = 0.5


def listed():
    return [
        # one token between two blocks of a decoder (hidden size of the o_proj benchmark)
        {"name": "norm_fwd_m1_d8192", "op": "norm_fwd", "M": 1, "D": 8192, "gate_rows": 1},
        # a prompt or training step of the o_proj benchmark, a gate row for each of 4 sequences
        {"name": "norm_fwd_m2048_d8192", "op": "norm_fwd", "M": 2048, "D": 8192, "gate_rows": 4},
        # a training batch of the down_proj benchmark, a gate value for each channel
        {"name": "norm_bwd_m8192_d8192", "op": "norm_bwd", "M": 8192, "D": 8192, "gate_rows": 1},
        # odd sizes, a gate value for each element
        {"name": "norm_bwd_m1003_d6152", "op": "norm_bwd", "M": 1003, "D": 6152, "gate_rows": 1003},
        # the input of the down_proj layer kept and restored: smallest and largest batch of its benchmark
        {"name": "act8_m512_k28672", "op": "act8", "M": 512, "K": 28672},
        {"name": "act8_m8192_k28672", "op": "act8", "M": 8192, "K": 28672},
        # backward pass of the o_proj layer, of the down_proj layer with few tokens, and of a ragged one
        {"name": "backward_m2048_n8192_k8192", "op": "backward", "M": 2048, "N": 8192, "K": 8192},
        {"name": "backward_m512_n8192_k28672", "op": "backward", "M": 512, "N": 8192, "K": 28672},
        {"name": "backward_m392_n776_k1600", "op": "backward", "M": 392, "N": 776, "K": 1600},
        # one token through o_proj, one through down_proj (weights with zero points)
        {"name": "w4_m1_n8192_k8192", "op": "w4", "M": 1, "N": 8192, "K": 8192, "group": 128, "zeros": False},
        {"name": "w4_m1_n8192_k28672", "op": "w4", "M": 1, "N": 8192, "K": 28672, "group": 128, "zeros": True},
        # a batch of 16 tokens through the 6144 x 16384 expert's down_proj, small groups
        {"name": "w4_m16_n6144_k16384", "op": "w4", "M": 16, "N": 6144, "K": 16384, "group": 64, "zeros": False},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "act8", "backward", "w4"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 64, 12288, 8)
        gate = rng.choice(["none", "channel", "sequence", "element"])
        M = _log(rng, 1, min(32768, 8192 * 8192 // D))
        gate_rows = {"none": 0, "channel": 1, "element": M}.get(gate)
        if gate_rows is None:
            gate_rows = rng.choice([2, 4, 7])
            M = gate_rows * max(1, M // gate_rows)
        return {"op": op, "M": M, "D": D, "gate_rows": gate_rows}
    if op == "act8":
        K = _log(rng, 512, 28672, 64)
        return {"op": op, "M": _log(rng, 8, min(32768, 8192 * 28672 // K), 8), "K": K}
    if op == "backward":
        N, K = _log(rng, 64, 12288, 8), _log(rng, 512, 28672, 64)
        return {"op": op, "M": _log(rng, 8, max(8, min(8192, 2048 * 8192 * 8192 // (N * K))), 8), "N": N, "K": K}
    N, K = _log(rng, 256, 12288, 8), _log(rng, 1024, 28672, 64)
    if N * K > 8192 * 28672:
        N = 8192
    return {"op": op, "M": _log(rng, 1, 32), "N": N, "K": K, "group": rng.choice([32, 64, 128]),
            "zeros": rng.choice([False, True])}


def _gate_of(case, normal):
    g = case["gate_rows"]
    return (0.3 * normal(g, case["D"]) + 0.5).to(torch.bfloat16) if g else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def activations(*shape):
        """N(0, 1) with 5% of the entries scaled by 8, as after a gated activation."""
        a = normal(*shape).to(torch.bfloat16)
        out = torch.rand(*shape, generator=gen, device="cuda", dtype=torch.bfloat16) < 0.05
        return torch.where(out, a * 8, a)

    op, bf16 = case["op"], torch.bfloat16
    s = {"case": case, "own": own}
    if op in ("norm_fwd", "norm_bwd"):
        M, D = case["M"], case["D"]
        # a residual stream with some strong channels, and a block output of unit variance
        s["x"] = (normal(M, D) * (1 + 4 * (normal(D).abs() > 2.5))).to(bf16)
        s["y"] = normal(M, D).to(bf16)
        s["w_post"] = (1 + 0.1 * normal(D)).to(bf16)
        s["w_pre"] = (1 + 0.1 * normal(D)).to(bf16)
        s["gate"] = _gate_of(case, normal)
        if op == "norm_bwd":
            s["dr"] = (0.02 * normal(M, D)).to(bf16)
            s["dh"] = (0.02 * normal(M, D)).to(bf16)
            s["stats"] = _norm_forward(s)[2]  # what the forward pass kept
        if own:
            from tensor_gemm_reduce_gb300 import block_norm
            if op == "norm_fwd":
                s["out"] = block_norm.new_outputs(s["x"])
            else:
                s["out"] = block_norm.new_gradients(s["x"], s["gate"])
                s["ws"] = block_norm.new_workspace(s["x"], s["gate"])
    elif op == "act8":
        s["A"] = activations(WORLD, case["M"], case["K"] // WORLD)
        if own:
            from tensor_gemm_reduce_gb300 import act8
            s["ck"] = act8.Checkpoint(case["M"], case["K"])
            s["out"] = torch.empty_like(s["A"])
    elif op == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        A = activations(WORLD, M, K // WORLD)
        s["W"] = (normal(WORLD, K // WORLD, N) * K ** -0.5).to(bf16)
        s["dY"] = (0.02 * normal(M, N)).to(bf16)
        if own:
            from tensor_gemm_reduce_gb300 import act8
            s["ck"] = act8.save(A)
            s["plan"] = act8.BackwardPlan(M, N, K)
            s["ws"] = s["plan"].new_workspace()
            s["dA"], s["dW"] = torch.empty_like(A), torch.empty_like(s["W"])
        else:
            s["q"], s["e"] = _save8(A)
    else:
        M, N, K, g = case["M"], case["N"], case["K"], case["group"]
        Kr = K // WORLD
        G = -(-Kr // g)
        s["x"] = activations(WORLD, M, Kr)
        codes = torch.empty(WORLD, Kr, N, dtype=torch.uint8, device="cuda")
        for r in range(WORLD):
            codes[r] = ((normal(Kr, N) * 2.7).round() + 8).clamp(0, 15).to(torch.uint8)
        scales = ((0.5 + torch.rand(WORLD, G, N, generator=gen, device="cuda")) * K ** -0.5 / 2.7).to(bf16)
        zeros = None
        if case["zeros"]:
            zeros = torch.randint(5, 12, (WORLD, G, N), generator=gen, device="cuda", dtype=torch.uint8)
        if own:
            from tensor_gemm_reduce_gb300 import w4
            s["weight"] = w4.pack(codes, scales, zeros, group=g)
            s["ws"] = w4.new_workspace(s["weight"])
            s["out"] = torch.empty(M, N, dtype=bf16, device="cuda")
        else:
            s["codes"], s["scales"], s["zeros"] = codes, scales, zeros
    return s


# ---------------------------------------------------------------- plain forms


def _gate_rows(gate, M):
    """[G][D] as a factor that broadcasts over [G][M/G][D]."""
    return gate.float()[:, None, :] if gate is not None else torch.ones(1, 1, 1, device="cuda")


def _norm_forward(s):
    x, y = s["x"].float(), s["y"].float()
    M, D = x.shape
    G = s["case"]["gate_rows"] or 1
    p = 1 / torch.sqrt((y * y).mean(1) + EPS)
    u = y * p[:, None] * s["w_post"].float()
    r = x + SCALE * (_gate_rows(s["gate"], M) * u.view(G, M // G, D)).view(M, D)
    q = 1 / torch.sqrt((r * r).mean(1) + EPS)
    h = r * q[:, None] * s["w_pre"].float()
    return r.to(torch.bfloat16), h.to(torch.bfloat16), torch.stack([p, q])


def _norm_backward(s):
    bf16 = torch.bfloat16
    x, y, dr, dh = s["x"].float(), s["y"].float(), s["dr"].float(), s["dh"].float()
    w_post, w_pre = s["w_post"].float(), s["w_pre"].float()
    p, q = s["stats"][0][:, None], s["stats"][1][:, None]
    M, D = x.shape
    G = s["case"]["gate_rows"] or 1
    g = (_gate_rows(s["gate"], M) * SCALE).expand(G, M // G, D).reshape(M, D)
    yn = y * p
    rn = (x + g * yn * w_post) * q
    a = dh * w_pre
    t = dr + q * (a - rn * (a * rn).mean(1, keepdim=True))
    v = g * t
    b = v * w_post
    dy = p * (b - yn * (b * yn).mean(1, keepdim=True))
    out = {"dx": t.to(bf16), "dy": dy.to(bf16), "dw_post": (v * yn).sum(0).to(bf16),
           "dw_pre": (dh * rn).sum(0).to(bf16)}
    if s["gate"] is not None:
        out["dgate"] = (SCALE * t * yn * w_post).view(G, M // G, D).sum(1).to(bf16)
    return out


def _save8(A):
    """int8 codes and exponents of groups of GROUP8 along the last axis."""
    a = A.float()
    n = a.shape[-1]
    a = torch.nn.functional.pad(a, (0, -n % GROUP8)).unflatten(-1, (-1, GROUP8))
    m, ex = torch.frexp(a.abs().amax(-1))
    e = (ex - 7 + (m > 127 / 128)).clamp(min=-126)
    q = torch.round(torch.ldexp(a, -e[..., None])).to(torch.int8)
    return q.flatten(-2)[..., :n], e


def _restore8(q, e):
    return torch.ldexp(q.float(), e.repeat_interleave(GROUP8, -1)[..., :q.shape[-1]])


def _plain(s):
    op, bf16 = s["case"]["op"], torch.bfloat16
    if op == "norm_fwd":
        r, h, stats = _norm_forward(s)
        return {"r": r, "h": h, "stats": stats}
    if op == "norm_bwd":
        return _norm_backward(s)
    if op == "act8":
        return _restore8(*_save8(s["A"])).to(bf16)
    if op == "backward":
        dY, W, A = s["dY"].float(), s["W"].float(), _restore8(s["q"], s["e"])
        return {"dA": torch.matmul(dY, W.transpose(1, 2)).to(bf16),
                "dW": torch.matmul(A.transpose(1, 2), dY).to(bf16)}
    g, Kr = s["case"]["group"], s["codes"].shape[1]

    def rows(t):
        return t.float().repeat_interleave(g, 1)[:, :Kr]

    zero = 8.0 if s["zeros"] is None else rows(s["zeros"])
    w = (s["codes"].float() - zero) * rows(s["scales"])
    return torch.matmul(s["x"].float(), w).sum(0).to(bf16)


def run(s):
    if not s["own"]:
        return _plain(s)
    op = s["case"]["op"]
    if op == "norm_fwd":
        from tensor_gemm_reduce_gb300 import block_norm
        r, h, stats = block_norm.forward(s["x"], s["y"], s["w_post"], s["w_pre"], gate=s["gate"],
                                         scale=SCALE, eps=EPS, out=s["out"])
        return {"r": r, "h": h, "stats": stats}
    if op == "norm_bwd":
        from tensor_gemm_reduce_gb300 import block_norm
        dx, dy, dw_post, dw_pre, dgate = block_norm.backward(
            s["dr"], s["dh"], s["x"], s["y"], s["w_post"], s["w_pre"], s["stats"], gate=s["gate"],
            scale=SCALE, out=s["out"], workspace=s["ws"])
        out = {"dx": dx, "dy": dy, "dw_post": dw_post, "dw_pre": dw_pre}
        if dgate is not None:
            out["dgate"] = dgate
        return out
    if op == "act8":
        from tensor_gemm_reduce_gb300 import act8
        return act8.restore(act8.save(s["A"], out=s["ck"]), out=s["out"])
    if op == "backward":
        s["plan"].run(s["dY"], s["W"], s["ck"], s["dA"], s["dW"], s["ws"])
        return {"dA": s["dA"], "dW": s["dW"]}
    from tensor_gemm_reduce_gb300 import w4
    return w4.matvec(s["x"], s["weight"], out=s["out"], workspace=s["ws"])


def work(case):
    op, M = case["op"], case["M"]
    if op in ("norm_fwd", "norm_bwd"):
        D, g = case["D"], case["gate_rows"]
        if op == "norm_fwd":  # x, y -> r, h, and the row statistics
            return {"bytes": 8 * M * D + 2 * g * D + 4 * D + 8 * M, "flops": 12 * M * D}
        return {"bytes": 12 * M * D + 4 * g * D + 8 * D + 8 * M, "flops": 30 * M * D}
    K = case["K"]
    kept = M * K + M * K // GROUP8  # codes and exponents
    if op == "act8":  # written by save, read by restore
        return {"bytes": 4 * M * K + 2 * kept, "flops": 4 * M * K}
    N = case["N"]
    if op == "backward":
        return {"bytes": 2 * M * N + 4 * K * N + kept + 2 * M * K, "flops": 4 * M * N * K}
    groups = WORLD * -(-(K // WORLD) // case["group"])
    per_group = 2.5 if case["zeros"] else 2
    return {"bytes": int(N * K // 2 + per_group * groups * N + 2 * M * K + 2 * M * N), "flops": 2 * M * N * K}


# ---------------------------------------------------------------- in 64 bits


def _exact_norm(s, backward):
    leaf = {k: s[k].double().requires_grad_(backward) for k in ("x", "y", "w_post", "w_pre")}
    x, y = leaf["x"], leaf["y"]
    gate = s["gate"].double().requires_grad_(backward) if s["gate"] is not None else None
    M = x.shape[0]
    p = torch.rsqrt(y.square().mean(-1) + EPS)
    branch = torch.einsum("md,m,d->md", y, p, leaf["w_post"]) * SCALE
    if gate is not None:
        branch = branch * gate.repeat_interleave(M // gate.shape[0], 0)
    r = x + branch
    q = torch.rsqrt(r.square().mean(-1) + EPS)
    h = torch.einsum("md,m,d->md", r, q, leaf["w_pre"])
    if not backward:
        return {"r": r, "h": h, "stats": torch.stack([p, q])}
    wanted = [x, y, leaf["w_post"], leaf["w_pre"]] + ([gate] if gate is not None else [])
    grads = torch.autograd.grad([r, h], wanted, [s["dr"].double(), s["dh"].double()])
    return dict(zip(["dx", "dy", "dw_post", "dw_pre", "dgate"], grads))


def _exact8(A):
    """The value a checkpoint stands for: the scale is the first of the powers of two whose 127-fold holds the group."""
    n = A.shape[-1]
    a = torch.nn.functional.pad(A.double(), (0, -n % GROUP8)).unflatten(-1, (-1, GROUP8))
    powers = torch.pow(2.0, torch.arange(-126, 123, dtype=torch.float64, device=A.device))
    scale = powers[torch.searchsorted(127 * powers, a.abs().amax(-1, keepdim=True).contiguous())]
    return (torch.round(a / scale) * scale).flatten(-2)[..., :n]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s, op == "norm_bwd")
    if op == "act8":
        return _exact8(s["A"])
    if op == "backward":
        A = s["q"].double() * torch.pow(2.0, s["e"].double()).repeat_interleave(GROUP8, -1)[..., :s["q"].shape[-1]]
        dY = s["dY"].double()
        return {"dA": torch.einsum("mn,rkn->rmk", dY, s["W"].double()),
                "dW": torch.einsum("rmk,mn->rkn", A, dY)}
    total = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    g, Kr = case["group"], case["K"] // WORLD
    for r in range(WORLD):
        group_of = torch.arange(Kr, device="cuda") // g
        zero = s["zeros"][r].double()[group_of] if s["zeros"] is not None else 8.0
        total += s["x"][r].double() @ ((s["codes"][r].double() - zero) * s["scales"][r].double()[group_of])
    return total
