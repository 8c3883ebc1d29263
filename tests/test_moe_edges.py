"""Routing and the experts' layer where scores saturate, logits are not finite, choices tie at the
border and tensors are empty in part, against the definitions in float64.

Tolerances.  A routed weight is a quotient of exponentials of fp32 differences: an exponential is off
by 2 units in the last place, 4 * 2**-24, its argument x by |x| * 2**-24; a score takes two of them, a sum
and a quotient, the sum of up to 16 another 16 roundings: below 64 * 2**-24 of it for |x| up to 16, and in
all 64 + |x|.  A sigmoid's gradient takes the complement of a score as well, two exponentials and two
roundings more: 96 * 2**-24 of the terms that it is the difference of.
"""
import pytest
import torch

from tensor_gemm_reduce_gb300 import fp8, moe
from tensor_gemm_reduce_gb300 import gemm_rs as G
from test_fp8 import U, bits
from test_moe import assert_arranged, call, chosen, experts, order

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def shares(logits, ids):
    """The chosen sigmoids' shares of their sum, in float64 without underflow."""
    l = logits.double().gather(1, ids.long())
    return torch.softmax(-torch.nn.functional.softplus(-l), 1)


def by_logits(logits, p, k, groups, top_groups):
    best = p.unflatten(1, (groups, -1)).sort(-1, descending=True).values[..., :2].sum(-1)
    kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :top_groups]
    stays = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(logits.shape[1] // groups, 1)
    left = torch.where(stays, logits.double(), -1e300)  # below every logit here but a NaN's -inf
    left = torch.where(stays & torch.isneginf(logits), -1e299, left)
    return torch.sort(left, dim=1, descending=True, stable=True).indices[:, :k].int()


LOW = [(3, 8, 2), (300, 8, 2), (300, 40, 6), (40, 200, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", LOW)
def test_sigmoids_below_the_least_of_fp32(T, E, k):
    """Scores whose exponentials overflow have their ratio."""
    g = torch.Generator().manual_seed(T + E)
    logits = -90 - 4 * torch.rand(T, E, generator=g) - 100 * (torch.arange(T)[:, None] % 5)
    logits[1, 1:] = -torch.inf  # one score alone
    o = dict(score="sigmoid", scale=1.5)
    r = call(logits, k, o)
    ids = chosen(logits, k)[0]  # the logits' order
    assert torch.equal(r.ids.cpu(), ids)
    p = shares(logits, ids)
    p[1] = torch.eye(k)[0]
    assert ((r.weights.cpu().double() - 1.5 * p).abs() <= 64 * U * 1.5 * p).all()
    dw = torch.randn(T, k, generator=g)
    got = moe.route_backward(dw.cuda(), logits.cuda(), r).cpu().double()
    d, grad = 1.5 * dw.double(), torch.zeros(T, E, dtype=torch.float64)
    bound = torch.zeros_like(grad)
    mean, mag = (d * p).sum(1, keepdim=True), (d.abs() * p).sum(1, keepdim=True)
    grad.scatter_(1, ids.long(), p * (d - mean))
    bound.scatter_(1, ids.long(), 96 * U * p * (d.abs() + mag))
    assert ((got - grad).abs() <= bound + 1e-38).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", LOW)
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_saturated_sigmoids(T, E, k, renormalize):
    """The complement of a score near 1 is not what is left of it in fp32."""
    g = torch.Generator().manual_seed(T)
    logits = torch.tensor([8.0, -8, 10, 12, -10, 15, 17, 20, -20, 25, 30, 0])[torch.randint(0, 12, (T, E), generator=g)]
    logits += 0.5 * torch.rand(T, E, generator=g)
    logits[0] = 15 + torch.arange(E) / 64
    scale = 1.0 if renormalize else 2.5
    r = call(logits, k, dict(score="sigmoid", renormalize=renormalize, scale=scale))
    ids = r.ids.cpu().long()
    # the logits' order, which float64 no longer sees in scores this near 1
    assert torch.equal(ids, torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k])
    dw = torch.randn(T, k, generator=g)
    got = moe.route_backward(dw.cuda(), logits.cuda(), r).cpu().double()
    l, d = logits.double().gather(1, ids), scale * dw.double()
    rest = torch.sigmoid(-l)
    if renormalize:
        p = shares(logits, ids)
        want, mag = p * (d - (d * p).sum(1, keepdim=True)) * rest, p * (d.abs() + (d.abs() * p).sum(1, keepdim=True)) * rest
    else:
        want = d * torch.sigmoid(l) * rest
        mag = want.abs()
    grad = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, want)
    bound = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, 96 * U * mag)
    assert ((got - grad).abs() <= bound + 1e-38).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(8, 40), (300, 40), (300, 200), (40, 200)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_choice_beside_logits_that_are_not_finite(T, E, score):
    """A NaN counts as the lowest logit, +inf takes a softmax whole; neither touches the order of the others."""
    g = torch.Generator().manual_seed(T + E)
    logits, bias = torch.randn(T, E, generator=g), 0.2 * torch.randn(E, generator=g)
    logits[0, E - 1] = torch.nan
    logits[1, E - 1] = torch.inf
    logits[2, [0, E - 2]] = torch.inf
    logits[3, [E - 3, 5]] = torch.nan
    logits[4, [3, E - 4]] = torch.tensor([torch.nan, torch.inf])
    clean = torch.where(logits.isnan(), -torch.inf, logits)
    top = clean.max(1, keepdim=True).values
    # scores as the definition's limit, for the oracle: of 2000 in place of an infinity the rest's are 0
    finite = torch.where(torch.isposinf(clean), 2000.0, clean) if score == "softmax" else clean
    k = 4
    for o in (dict(groups=5, top_groups=2), dict(groups=4, top_groups=1), dict(bias=bias), dict(groups=5, top_groups=2, bias=bias)):
        for renormalize in (True, False):
            opts = {n: v for n, v in o.items() if n != "bias"}
            r = call(logits, k, dict(opts, score=score, renormalize=renormalize), o.get("bias"))
            ids, p = chosen(finite, k, o.get("bias"), score, opts.get("groups", 1), opts.get("top_groups"))
            if "bias" not in o:  # then experts of the groups that stay are compared by their logits
                ids = by_logits(clean, p, k, **opts)
            assert torch.equal(r.ids.cpu(), ids)
            w = r.weights.cpu()
            nan = logits.isnan().any(1)
            assert w[nan].isnan().all()
            rest = torch.where(ids >= 0, p.gather(1, ids.long()), 0)
            want = rest / rest.sum(1, keepdim=True) if renormalize else rest
            assert ((w.double() - want).abs() <= (64 + 16) * U * want + 1e-38)[~nan].all()
            d = moe.route_backward(torch.ones(T, k).cuda(), logits.cuda(), r).cpu()
            assert d[nan].isnan().all() and d[~nan].isfinite().all()
    assert top[1] == torch.inf


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(3, 12), (300, 12), (300, 96), (300, 200), (30, 200)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_choices_at_the_border_hide_no_better_one(T, E, score):
    """The last that is chosen and the first that is not are equal, and a third is above both by less than fp32 tells."""
    g = torch.Generator().manual_seed(E)
    bias = torch.ones(E)
    logits = torch.randint(-22, -18, (T, E), generator=g).float()
    logits[:, 0] = 0
    logits[0] = torch.full((E,), -40.0)
    logits[0, :4] = torch.tensor([0.0, -20, -20, -19])
    for k in (2, 3, 7):
        ids, _ = chosen(logits, k, bias, score)
        if T > 3:
            assert (ids[:, 1] != 1).any()
        assert torch.equal(call(logits, k, dict(score=score), bias).ids.cpu(), ids)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [40, 96, 128, 200, 256])
def test_nearly_equal_softmax_scores_of_many_experts(E):
    """Biases that make up for one token's scores up to their rounding; the others' logits are a little off it."""
    g = torch.Generator().manual_seed(E)
    base = torch.randn(1, E, generator=g)
    bias = (0.3 - chosen(base, 1)[1][0]).float()
    for spread in (1e-7, 3e-6, 3e-5):
        logits = base + spread * torch.randn(600, E, generator=g)
        for T in (600, 20):
            ids, _ = chosen(logits[:T], 6, bias)
            assert torch.equal(call(logits[:T].contiguous(), 6, {}, bias).ids.cpu(), ids)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(6, 8, 2), (300, 40, 6), (40, 200, 3)])
def test_masked_tokens_of_any_logits_have_no_gradient(T, E, k):
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(T))
    for t, v in enumerate((torch.nan, torch.inf, -torch.inf)):
        logits[t, 1] = v
    logits[3] = torch.nan
    mask = torch.arange(T) > 3
    for o in (dict(), dict(renormalize=False), dict(score="sigmoid"), dict(score="sigmoid", renormalize=False)):
        r = call(logits, k, o, mask=mask)
        assert (r.ids[:4] == -1).all() and (r.weights[:4] == 0).all()
        d = moe.route_backward(torch.ones(T, k).cuda(), logits.cuda(), r).cpu()
        assert (d[:4] == 0).all() and d.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 200])
def test_an_empty_contraction_leaves_the_rows_behind_the_last(T):
    E, k, K = 4, 2, 512
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(T), dtype=I32)
    ids[::3] = -1
    r = moe.arrange(ids.cuda(), torch.ones(T, k).cuda(), E)
    used = int(r.offsets[-1])
    assert 0 < used < T * k
    weight = fp8.quantize(torch.empty(E, 8, K // 8, 0, dtype=BF16, device="cuda"))
    ck, ws = moe.Checkpoint(r, weight), moe.new_workspace(r, weight)
    moe.forward(torch.zeros(8, T * k, K // 8, dtype=BF16, device="cuda"), weight, r, checkpoint=ck)
    dA = torch.full((8, T * k, K // 8), 3.0, dtype=BF16, device="cuda")
    dw = torch.full((T, k), 3.0, device="cuda")
    moe.backward(torch.empty(T, 0, dtype=BF16, device="cuda"), weight, r, ck, out=(dA, None, dw), workspace=ws)
    assert fp8.status(ws) == G.GEMM_RS_OK
    assert (dA[:, :used] == 0).all() and (dA[:, used:] == 3).all() and (dw == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 150])
@pytest.mark.parametrize("scales", [torch.float32, torch.float8_e8m0fnu])
def test_a_pair_outside_the_tensors_takes_nothing_of_the_first_token(T, scales):
    E, k, N, K = 3, 2, 136, 1088
    ids, w, A, W, dout = experts(T, E, k, N, K, False)
    ids[0] = -1  # a padded token, whose gradient is anything
    dout[0] = torch.nan
    weight, r = fp8.quantize(W.cuda(), scales=scales), moe.arrange(ids.cuda(), w.cuda(), E)
    ck = moe.Checkpoint(r, weight)
    moe.forward(A.cuda(), weight, r, checkpoint=ck)
    used = int(r.offsets[-1])
    r.pairs[3] = 1 << 30
    dA, dW, _ = moe.backward(dout.cuda(), weight, r, ck)
    assert not dA[:, 3].any() and dA[:, :used].isfinite().all() and dW.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(65536, 96, 6), (45000, 128, 7), (34001, 256, 8), (40000, 33, 8), (70001, 70, 4),
                                   (49999, 32, 7)])
def test_many_pairs_of_many_experts(T, E, k):
    """More than 262144 pairs and 32 experts or more: each number of CTAs that share an expert's ids."""
    ids = torch.randint(-1, E + 1, (T, k), generator=torch.Generator().manual_seed(T), dtype=I32)
    ids[T // 3:T // 2] = 5  # many of one
    r = moe.Routing(T, k, E)
    r.pairs.fill_(-7)
    moe.arrange(ids.cuda(), torch.rand(T, k).cuda(), E, out=r)
    assert_arranged(r, ids)
    assert (r.pairs[int(r.offsets[-1]):] == -7).all()


@pytest.mark.gpu
def test_the_places_of_a_padded_batch_are_indices():
    """x[pairs // k], as the module's documentation has it, with masked tokens."""
    taken = torch.full((1 << 20,), 1 << 30, dtype=I32, device="cuda")
    del taken  # the allocator's memory, of which the routing is made
    T, E, k = 1000, 8, 2
    x, mask = bits(T, 64).cuda(), torch.arange(T) % 3 > 0
    r = call(torch.randn(T, E, generator=torch.Generator().manual_seed(1)), k, {}, mask=mask)
    assert ((r.pairs >= 0) & (r.pairs < T * k)).all()
    used = int(r.offsets[-1])
    rows, _, pairs = order(r.ids.cpu(), E)
    assert torch.equal(x[r.pairs.long() // k][:used].cpu(), x.cpu()[pairs.long() // k])


# ---------------------------------------------------------------- no GPU needed


def test_a_new_routing_holds_places_of_the_tensors(monkeypatch):
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *s, **kw: empty(*s, **kw).fill_(1 << 20))
    r = moe.Routing(5, 2, 4, device="cpu")
    assert ((r.pairs >= 0) & (r.pairs < 10)).all()


@pytest.mark.parametrize("scales", [torch.float32, torch.float8_e8m0fnu])
@pytest.mark.parametrize("N,K,experts", [(0, 512, None), (0, 512, 3), (16, 0, None), (0, 0, 2)])
def test_loading_a_weight_of_nothing(N, K, experts, scales):
    weight = fp8.Weight(N, K, experts, device="cpu", scales=scales)
    codes = torch.zeros(weight.shape).to(torch.float8_e4m3fn)
    assert weight.load(codes, torch.zeros(weight.scales.shape).to(scales)) is weight
    assert weight.codes.shape == weight.shape
