"""Routing to experts, and the row-parallel layer in 8-bit floating point, for
one weight and for the weights of several experts, as they are measured.

route: scores, choice and weights of each token's experts, the order of the
token-expert pairs by expert, and the gradient of the scores; layer: out =
sum_r A_r W_r in e4m3 with a scale for each block of 128, forward and backward;
experts: the same product for each expert's tokens, weighted and summed for each
token.  M tokens (T where they are routed), N output columns, K inner dimension
over 8 virtual ranks, E experts, k of them for a token.
"""
import math

import torch

own = False

WORLD = 8
BLOCK = 128
LARGEST = 448.0  # of e4m3
SMALLEST = 2.0 ** -100  # a block's largest magnitude counts as at least this
SCALE = 1.5  # of the routed weights where they are not renormalised


def listed():
    return [
        # one token of a decoder chooses 2 of the 8 experts of the 6144 x 16384 mixture
        {"name": "route_t1_e8", "op": "route", "T": 1, "E": 8, "k": 2, "type": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "renormalize": True, "masked": False, "train": False},
        # its training batch, with the gradient of the scores
        {"name": "route_train_t2048_e8", "op": "route", "T": 2048, "E": 8, "k": 2, "type": "fp32",
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renormalize": True, "masked": False,
         "train": True},
        # prompts of a mixture of many small experts: balanced by a bias, experts in groups, a padded batch
        {"name": "route_t16384_e96", "op": "route", "T": 16384, "E": 96, "k": 6, "type": "fp32", "score": "sigmoid",
         "bias": True, "groups": 6, "top_groups": 3, "renormalize": True, "masked": True, "train": False},
        # one token through the down_proj layer, a serving batch through o_proj
        {"name": "layer_m1_n8192_k28672", "op": "layer", "M": 1, "N": 8192, "K": 28672, "train": False},
        {"name": "layer_m24_n8192_k8192", "op": "layer", "M": 24, "N": 8192, "K": 8192, "train": False},
        # prompts through both, the batches of their benchmarks
        {"name": "layer_m2048_n8192_k8192", "op": "layer", "M": 2048, "N": 8192, "K": 8192, "train": False},
        {"name": "layer_m8192_n8192_k28672", "op": "layer", "M": 8192, "N": 8192, "K": 28672, "train": False},
        # training steps: ragged sizes, and the batch of the o_proj benchmark
        {"name": "layer_train_m392_n776_k1600", "op": "layer", "M": 392, "N": 776, "K": 1600, "train": True},
        {"name": "layer_train_m2048_n8192_k8192", "op": "layer", "M": 2048, "N": 8192, "K": 8192, "train": True},
        # the mixture's experts: one token, a training step of its benchmark's batch
        {"name": "experts_t1_e8_n6144_k16384", "op": "experts", "T": 1, "E": 8, "k": 2, "N": 6144, "K": 16384,
         "masked": False, "train": False},
        {"name": "experts_train_t2048_e8_n6144_k16384", "op": "experts", "T": 2048, "E": 8, "k": 2, "N": 6144,
         "K": 16384, "masked": False, "train": True},
        # a padded batch through few experts of odd sizes
        {"name": "experts_train_t203_e5_n1032_k2624", "op": "experts", "T": 203, "E": 5, "k": 3, "N": 1032, "K": 2624,
         "masked": True, "train": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    op = rng.choice(["route", "layer", "layer", "experts", "experts"])
    train = rng.choice([False, True])
    if op == "route":
        E = rng.choice([5, 8, 12, 16, 32, 60, 64, 96, 128, 192, 256])
        k = rng.randint(2, min(8, E))
        score = rng.choice(["softmax", "sigmoid"])
        fits = [g for g in (2, 3, 4, 6, 8, 12) if E % g == 0 and E // g >= 2]
        groups = rng.choice(fits) if fits and rng.random() < 0.5 else 1
        least = -(-k // (E // groups))  # groups that hold k experts
        return {"op": op, "T": _log(rng, 1, min(32768, 16384 * 96 // E)), "E": E, "k": k,
                "type": rng.choice(["bf16", "fp32"]), "score": score, "bias": rng.choice([False, True]),
                "groups": groups, "top_groups": rng.randint(least, groups), "renormalize": rng.choice([False, True]),
                "masked": rng.choice([False, True]), "train": train}
    if op == "layer":
        N, K = _log(rng, 64, 12288, 8), _log(rng, 512, 28672, 64)
        most = 2048 * 8192 * 8192 if train else 8192 * 8192 * 28672
        return {"op": op, "M": _log(rng, 1, max(1, min(8192, most // (N * K)))), "N": N, "K": K, "train": train}
    E = rng.choice([2, 4, 5, 8, 16])
    k = rng.randint(2, min(4, E))
    N, K = _log(rng, 64, 8192, 8), _log(rng, 512, 16384, 64)
    if E * N * K > 8 * 6144 * 16384:
        N = max(64, 8 * 6144 * 16384 // (E * K) // 8 * 8)
    T = _log(rng, 1, max(1, min(8192, 2 * 2048 * 6144 * 16384 // (k * N * K))))
    return {"op": op, "T": T, "E": E, "k": k, "N": N, "K": K, "masked": rng.choice([False, True]), "train": train}


def _options(case):
    return {"score": case["score"], "groups": case["groups"], "top_groups": case["top_groups"],
            "renormalize": case["renormalize"], "scale": 1.0 if case["renormalize"] else SCALE}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def activations(*shape):
        """N(0, 1) with 5% of the entries scaled by 8, as after a gated activation."""
        a = normal(*shape).to(bf16)
        out = torch.rand(*shape, generator=gen, device="cuda", dtype=bf16) < 0.05
        return torch.where(out, a * 8, a)

    def some(n):
        """Which of a padded batch's tokens count: all but about one in eight."""
        return torch.rand(n, generator=gen, device="cuda") >= 0.125 if case["masked"] else None

    op, train = case["op"], case["train"]
    s = {"case": case, "own": own}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # experts of unequal popularity
        logits = 1.5 * normal(T, E) + 0.5 * normal(E)
        s["logits"] = logits.to(bf16) if case["type"] == "bf16" else logits
        s["bias"] = 0.05 * normal(E) if case["bias"] else None
        s["mask"] = some(T)
        if train:
            s["dweights"] = 0.1 * normal(T, k)
        if own:
            from tensor_gemm_reduce_gb300 import moe
            s["routing"] = moe.Routing(T, k, E)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    N, K = case["N"], case["K"]
    Kr = K // WORLD
    if op == "layer":
        M = case["M"]
        s["A"] = activations(WORLD, M, Kr)
        W = (normal(WORLD, Kr, N) * K ** -0.5).to(bf16)
        if train:
            s["dY"] = (0.02 * normal(M, N)).to(bf16)
    else:
        T, E, k = case["T"], case["E"], case["k"]
        ids = (normal(T, E) + 0.3 * normal(E)).argsort(1, descending=True)[:, :k].int()
        weights = torch.softmax(normal(T, k), 1)
        mask = some(T)
        if mask is not None:
            ids[~mask] = -1
            weights[~mask] = 0
        s["ids"], s["weights"] = ids, weights
        s["counts"] = torch.bincount(ids[ids >= 0].long(), minlength=E).tolist()
        s["A"] = activations(WORLD, T * k, Kr)
        W = torch.empty(E, WORLD, Kr, N, dtype=bf16, device="cuda")
        for e in range(E):
            W[e] = (normal(WORLD, Kr, N) * K ** -0.5).to(bf16)
        if train:
            s["dY"] = (0.02 * normal(T, N)).to(bf16)
    if train:
        s["W"] = W  # a step quantises its weights anew
    if own:
        from tensor_gemm_reduce_gb300 import fp8, moe
        s["weight"] = fp8.quantize(W)
        s["out"] = torch.empty(case["M"] if op == "layer" else T, N, dtype=bf16, device="cuda")
        if op == "layer":
            s["ws"] = fp8.new_workspace(M, s["weight"])
            s["ck"] = fp8.Checkpoint(M, K) if train else None
            s["grads"] = fp8.new_gradients(M, s["weight"]) if train else None
        else:
            s["routing"] = moe.arrange(ids, weights, E)
            s["ws"] = moe.new_workspace(s["routing"], s["weight"])
            s["ck"], s["grads"] = None, None
            if train:
                s["ck"] = moe.Checkpoint(s["routing"], s["weight"])
                s["grads"] = moe.new_gradients(s["routing"], s["weight"])
                s["grads"][0].zero_()  # rows of dA behind the last token's are left as they were
    elif not train:
        s["codes"], s["scales"] = _codes(W, BLOCK, BLOCK)
    return s


# ---------------------------------------------------------------- plain forms


def _codes(x, rows, cols):
    """e4m3 codes of x's last two dimensions in blocks of rows x cols, padded to whole
    blocks [..., R, rows, C, cols], and the blocks' scales [..., R, 1, C, 1]."""
    r, c = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -c % cols, 0, -r % rows))
    x = x.unflatten(-1, (-1, cols)).unflatten(-3, (-1, rows)).float()
    scale = x.abs().amax((-3, -1), keepdim=True).clamp(min=SMALLEST) * (1 / LARGEST)
    return (x * scale.reciprocal()).to(torch.float8_e4m3fn), scale


def _values(codes, scales, shape):
    v = (codes.float() * scales).flatten(-2).flatten(-3, -2)
    return v[..., :shape[-2], :shape[-1]]


def _rounded(x, rows, cols):
    """x as its codes and scales stand for it."""
    return _values(*_codes(x, rows, cols), x.shape)


def _scores(logits, kind):
    # 64 bits: two experts' scores may differ by less than 32 bits tell apart
    return torch.softmax(logits.double(), -1) if kind == "softmax" else torch.sigmoid(logits.double())


def _order(ids, E):
    """(rows [T][k], offsets [E+1]) of the pairs in the order of their experts, then tokens."""
    flat = ids.flatten()
    chosen = flat >= 0
    order = torch.sort(torch.where(chosen, flat, E), stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), dtype=flat.dtype, device=flat.device)
    rows = torch.where(chosen, rows, -1).view(ids.shape)
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    return rows, torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()


def _plain_route(s):
    c, logits = s["case"], s["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    score = _scores(logits, c["score"])
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        g = choice.view(T, c["groups"], -1)
        best = g.sort(-1, descending=True).values[..., :2].sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        open_ = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(open_[..., None], g, -math.inf).view(T, E)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :k]
    p = score.gather(1, ids)
    o = _options(c)
    total = p.sum(1, keepdim=True) if c["renormalize"] else 1.0
    w = o["scale"] * p / total
    out_ids = ids.int()
    if s["mask"] is not None:
        out_ids = torch.where(s["mask"][:, None], out_ids, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    rows, offsets = _order(out_ids, E)
    out = {"ids": out_ids, "weights": w.float(), "rows": rows, "offsets": offsets}
    if c["train"]:
        dw = s["dweights"].double()
        if s["mask"] is not None:
            dw = torch.where(s["mask"][:, None], dw, 0.0)
        dp = o["scale"] / total * dw
        if c["renormalize"]:
            dp = dp - o["scale"] / total * (dw * p / total).sum(1, keepdim=True)
        ds = torch.zeros_like(score).scatter_(1, ids, dp)
        if c["score"] == "softmax":
            dl = score * (ds - (ds * score).sum(1, keepdim=True))
        else:
            dl = ds * score * (1 - score)
        out["dlogits"] = dl.to(logits.dtype)
    return out


def _by_token(A):
    """[8][M][K/8] as [M][K]."""
    return A.transpose(0, 1).flatten(1)


def _by_rank(x):
    return x.unflatten(1, (WORLD, -1)).transpose(0, 1)


def _plain_layer(s):
    c, bf16 = s["case"], torch.bfloat16
    shape = (WORLD, c["K"] // WORLD, c["N"])
    W = _values(*_codes(s["W"], BLOCK, BLOCK), shape) if c["train"] else _values(s["codes"], s["scales"], shape)
    W = W.flatten(0, 1)
    out = (_by_token(_rounded(s["A"], 1, BLOCK)) @ W).to(bf16)
    if not c["train"]:
        return out
    dA = _by_rank(_rounded(s["dY"], 1, BLOCK) @ W.t()).to(bf16)
    dW = _by_token(_rounded(s["A"], BLOCK, 1)).t() @ _rounded(s["dY"], BLOCK, 1)
    return {"out": out, "dA": dA, "dW": dW.unflatten(0, (WORLD, -1)).to(bf16)}


def _plain_experts(s):
    c, bf16 = s["case"], torch.bfloat16
    T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
    shape = (E, WORLD, K // WORLD, N)
    W = _values(*_codes(s["W"], BLOCK, BLOCK), shape) if c["train"] else _values(s["codes"], s["scales"], shape)
    W = W.flatten(1, 2)
    rows, offsets = _order(s["ids"], E)
    used, most = sum(s["counts"]), max(1, max(s["counts"]))  # rows that belong to a token, and an expert's most
    # row i of the sorted pairs is row at[i] of the experts' padded batches
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), offsets.diff(), output_size=used)
    at = expert * most + torch.arange(used, device="cuda") - offsets[expert]

    def padded(x):
        return torch.zeros(E * most, x.shape[1], device="cuda").index_copy_(0, at, x).view(E, most, -1)

    A = s["A"][:, :used]
    y = torch.bmm(padded(_by_token(_rounded(A, 1, BLOCK))), W).flatten(0, 1)[at]
    chosen = rows >= 0
    w = torch.where(chosen, s["weights"], 0.0)
    if used == 0:
        mine = torch.zeros(T, k, N, device="cuda")
    else:
        mine = torch.where(chosen[..., None], y[rows.clamp(min=0)], 0.0)
    out = (w[..., None] * mine).sum(1).to(bf16)
    if not c["train"]:
        return out
    dout = s["dY"].float()
    dweights = (dout[:, None] * mine).sum(-1)
    pair = torch.empty(used, dtype=torch.long, device="cuda")
    pair[rows[chosen].long()] = torch.arange(T * k, device="cuda").view(T, k)[chosen]
    dy = dout[pair // k] * w.flatten()[pair, None]
    dA = torch.zeros(T * k, K, device="cuda")
    dA[:used] = torch.bmm(padded(_rounded(dy, 1, BLOCK)), W.transpose(1, 2)).flatten(0, 1)[at]
    dW = torch.bmm(_rounded(padded(_by_token(A).float()), BLOCK, 1).transpose(1, 2), _rounded(padded(dy), BLOCK, 1))
    return {"out": out, "dA": _by_rank(dA).to(bf16), "dW": dW.view(shape).to(bf16), "dweights": dweights}


def run(s):
    c = s["case"]
    if not s["own"]:
        return {"route": _plain_route, "layer": _plain_layer, "experts": _plain_experts}[c["op"]](s)
    from tensor_gemm_reduce_gb300 import fp8, moe
    if c["op"] == "route":
        r = moe.route(s["logits"], c["k"], bias=s["bias"], mask=s["mask"], out=s["routing"], **_options(c))
        out = {"ids": r.ids, "weights": r.weights, "rows": r.rows, "offsets": r.offsets}
        if c["train"]:
            out["dlogits"] = moe.route_backward(s["dweights"], s["logits"], r, out=s["dlogits"])
        return out
    if c["train"]:
        fp8.quantize(s["W"], out=s["weight"])
    if c["op"] == "layer":
        out = fp8.forward(s["A"], s["weight"], checkpoint=s["ck"], out=s["out"], workspace=s["ws"])
        if not c["train"]:
            return out
        dA, dW = fp8.backward(s["dY"], s["weight"], s["ck"], out=s["grads"], workspace=s["ws"])
        return {"out": out, "dA": dA, "dW": dW}
    out = moe.forward(s["A"], s["weight"], s["routing"], checkpoint=s["ck"], out=s["out"], workspace=s["ws"])
    if not c["train"]:
        return out
    dA, dW, dweights = moe.backward(s["dY"], s["weight"], s["routing"], s["ck"], out=s["grads"], workspace=s["ws"])
    return {"out": out, "dA": dA, "dW": dW, "dweights": dweights}


def work(case):
    op, train = case["op"], case["train"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        item = 2 if case["type"] == "bf16" else 4
        # logits -> ids, weights and rows; backward: logits, ids and the weights' gradients -> the logits'
        return {"bytes": T * (E * item + 12 * k) + (T * (2 * E * item + 8 * k) if train else 0),
                "flops": T * E * (20 if train else 10)}
    N, K = case["N"], case["K"]
    if op == "layer":
        M, tokens, weights, extra = case["M"], case["M"], N * K, 0
    else:
        tokens = case["T"]
        M = tokens * case["k"]
        weights = N * K * (case["E"] if train else min(case["E"], M))
        extra = 16 * M
    if not train:
        return {"bytes": 2 * M * K + weights + 2 * tokens * N + extra, "flops": 2 * M * N * K}
    # W, A and dY -> the output, dA and dW
    return {"bytes": 4 * weights + 4 * M * K + 4 * tokens * N + extra, "flops": 6 * M * N * K}


# ---------------------------------------------------------------- in 64 bits


def _exact_rounded(x, rows, cols):
    """The values that x has in blocks of rows x cols: a scale of 32 bits, the least of e4m3's
    magnitudes' distances from x / scale, ties to the even one."""
    r, c = x.shape[-2:]
    R, C = -(-r // rows), -(-c // cols)
    full = torch.zeros(*x.shape[:-2], R * rows, C * cols, dtype=torch.float64, device=x.device)
    full[..., :r, :c] = x
    top = full.abs().unfold(-2, rows, rows).unfold(-2, cols, cols).amax((-2, -1)).clamp(min=SMALLEST)
    scale = top.float() * torch.tensor(1 / LARGEST, dtype=torch.float32, device=x.device)
    inverse = (1 / scale).double().repeat_interleave(rows, -2).repeat_interleave(cols, -1)
    scale = scale.double().repeat_interleave(rows, -2).repeat_interleave(cols, -1)
    v = (full * inverse).float().double()
    step = torch.pow(2.0, (torch.frexp(v).exponent - 1).clamp(min=-6).double() - 3)
    v = (torch.round(v / step) * step).clamp(-LARGEST, LARGEST)
    return (v * scale)[..., :r, :c]


def _exact_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].double().requires_grad_(c["train"])
    if c["score"] == "softmax":
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        p = 1 / (1 + torch.exp(-x))
    with torch.no_grad():
        choice = p.detach().clone()
        if s["bias"] is not None:
            choice += s["bias"].double()
        if c["groups"] > 1:
            size = E // c["groups"]
            best = choice.unfold(1, size, size).topk(2, -1).values.sum(-1)
            bar = best.topk(c["top_groups"], 1).values[:, -1:]
            choice[(best < bar).repeat_interleave(size, 1)] = -math.inf
        ids = choice.topk(k, 1).indices  # where scores tie this may choose another; whole numbers are not given
        ids = torch.where(choice.gather(1, ids) == choice.gather(1, ids).roll(-1, 1),
                          torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k], ids)
    w = torch.gather(p, 1, ids)
    w = w / w.sum(1, keepdim=True) if c["renormalize"] else w * SCALE
    if s["mask"] is not None:
        w = w * s["mask"][:, None]
    out = {"ids": None, "weights": w.detach(), "rows": None, "offsets": None}
    if c["train"]:
        out["dlogits"] = torch.autograd.grad(w, x, s["dweights"].double())[0]
    return out


def _exact_layer(s, W):
    A = s["A"].double()
    q = _exact_rounded(A, 1, BLOCK)
    out = torch.einsum("rmk,rkn->mn", q, W)
    if not s["case"]["train"]:
        return out
    dY = s["dY"].double()
    return {"out": out, "dA": torch.einsum("mn,rkn->rmk", _exact_rounded(dY, 1, BLOCK), W),
            "dW": torch.einsum("rmk,mn->rkn", _exact_rounded(A, BLOCK, 1), _exact_rounded(dY, BLOCK, 1))}


def _exact_experts(s, W):
    c = s["case"]
    T, E, k, N, Kr = c["T"], c["E"], c["k"], c["N"], c["K"] // WORLD
    f64 = {"dtype": torch.float64, "device": "cuda"}
    out, dweights = torch.zeros(T, N, **f64), torch.zeros(T, k, **f64)
    dA, dW = torch.zeros(WORLD, T * k, Kr, **f64), torch.zeros(E, WORLD, Kr, N, **f64)
    first = 0
    for e, n in enumerate(s["counts"]):
        if n == 0:
            continue
        token, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        A = s["A"][:, first:first + n].double()
        y = torch.einsum("rmk,rkn->mn", _exact_rounded(A, 1, BLOCK), W(e))
        weight = s["weights"][token, slot][:, None]
        out.index_add_(0, token, weight.double() * y)
        if c["train"]:
            d = s["dY"][token].double()
            dweights[token, slot] = (d * y).sum(1)
            d = (d.float() * weight).double()  # a pair's gradient is a product of 32 bits
            dA[:, first:first + n] = torch.einsum("mn,rkn->rmk", _exact_rounded(d, 1, BLOCK), W(e))
            dW[e] = torch.einsum("rmk,mn->rkn", _exact_rounded(A, BLOCK, 1), _exact_rounded(d, BLOCK, 1))
        first += n
    return {"out": out, "dA": dA, "dW": dW, "dweights": dweights} if c["train"] else out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "route":
        return _exact_route(s)
    shape = (WORLD, case["K"] // WORLD, case["N"])

    def weight(e=None):
        if case["train"]:
            return _exact_rounded((s["W"] if e is None else s["W"][e]).double(), BLOCK, BLOCK)
        at = (lambda t: t) if e is None else (lambda t: t[e])
        return _values(at(s["codes"]), at(s["scales"]).double(), shape).double()

    return _exact_layer(s, weight()) if case["op"] == "layer" else _exact_experts(s, weight)
