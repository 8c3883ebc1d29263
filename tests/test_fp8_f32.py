"""The layer and the experts' layer in 8-bit floating point with fp32 scales, the default: the tests
that test_fp8.py, test_moe.py and test_mixture.py hold of powers of two, with this form's definition,
and what the two forms have to say of each other.

Tolerance of a product: a step of 128 inner elements is four instructions on the tensor cores, each
of which adds 32 products of codes, which are exact, to the accumulator; each of its 33 addends may be
truncated where they are aligned, by 2**-23 of the largest, which is at most the sum of the absolute
terms: 4 * 33 * 2**-23.  Scaling a step takes the product of two scales, once more a column's own, and
the fused addition: 3 roundings of 2**-24, one to spare.  Steps are added up, 2**-24 each, at most
inner / 128 + 8 of them (each rank's last is ragged), then up to 8 parts of a contraction: 16 with one
to spare for each.  The result is rounded to bf16 once: 2**-8 of the value.
"""
import ctypes

import numpy as np
import pytest
import torch

import test_fp8
import test_moe
from tensor_gemm_reduce_gb300 import fp8, moe, ops_abi
from tensor_gemm_reduce_gb300 import gemm_rs as G
from test_fp8 import U, bits
from test_fp8 import test_backward, test_empty, test_every_token_count_gives_the_same_rows  # noqa: F401
from test_fp8 import test_few_tokens, test_forward, test_not_finite_values_stay_in_their_blocks  # noqa: F401
from test_fp8 import test_offsets_beyond_32_bits, test_powers_of_two_go_through  # noqa: F401
from test_fp8 import test_tensor_refusals  # noqa: F401
from test_mixture import test_a_block_against_the_formulas, test_memory_of_a_delayed_block_is_not_given_away  # noqa: F401
from test_mixture import test_two_graphs_with_one_workspace, test_two_streams_at_once  # noqa: F401
from test_moe import test_empty as test_empty_experts  # noqa: F401
from test_moe import test_experts_forward_and_backward, test_no_token_has_an_expert  # noqa: F401
from test_moe import test_not_finite_rows_stay_alone  # noqa: F401
from test_moe import test_offsets_beyond_32_bits as test_experts_offsets_beyond_32_bits  # noqa: F401
from test_moe import test_places_outside_the_tensors_are_passed_over  # noqa: F401
from test_moe import test_tensor_refusals as test_tensor_refusals_of_experts  # noqa: F401

BF16, F32, E8M0 = torch.bfloat16, torch.float32, torch.float8_e8m0fnu


def quantized(x, rows, cols):
    """(codes as float32 values, scales) of x's last two dimensions in blocks of rows x cols, on the CPU."""
    r, c = x.shape[-2:]
    x = torch.nn.functional.pad(x.float(), (0, -c % cols, 0, -r % rows)).unflatten(-1, (-1, cols)).unflatten(-3, (-1, rows))
    top = x.abs().amax((-3, -1), keepdim=True)
    scale = torch.where(top.isfinite(), top.clamp(min=2.0 ** -100) * torch.tensor(1 / 448, dtype=F32), torch.nan)
    q = (x * scale.reciprocal()).to(torch.float8_e4m3fn).float()
    return q.flatten(-2).flatten(-3, -2)[..., :r, :c], scale.double()


def assert_product(got, a, b, form, inner):
    ref, mag = np.einsum(form, a, b), np.einsum(form, abs(a), abs(b))
    got = got.double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(ref) + (4 * 33 * 2 + 4 + inner / 128 + 8 + 16) * U * mag + 1e-38
    err = np.abs(got - ref)
    assert np.isfinite(got).all() and (err <= bound).all(), f"worst {np.nanmax(err / bound):.2f} x the bound"


@pytest.fixture(autouse=True)
def this_form(monkeypatch):
    assert fp8.default_scales() is F32
    monkeypatch.setattr(test_fp8, "quantized", quantized)
    for module in (test_fp8, test_moe):
        monkeypatch.setattr(module, "assert_product", assert_product)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(8, 64), (136, 576), (520, 1600), (264, 8192)])
@pytest.mark.parametrize("low,high", [(0, 1), (-133, -95), (-30, 30), (100, 127)])
def test_weights_are_quantized_as_defined(N, K, low, high):
    g = torch.Generator().manual_seed(N + high)
    x = torch.randn(8, K // 8, N, generator=g).clamp(-1.9, 1.9)
    W = (x * torch.exp2(torch.randint(low, high, x.shape, generator=g).float())).to(BF16)
    W[1, :, :128] = 0  # a block of nothing
    weight = fp8.quantize(W.cuda())
    assert weight.scales.dtype is F32
    codes, scales = quantized(W, 128, 128)
    assert torch.equal(weight.codes.float().cpu(), codes)
    assert torch.equal(weight.scales.cpu().double(), scales.squeeze(-1).squeeze(-2))


@pytest.mark.gpu
def test_scales_made_elsewhere():
    """fp32 scales of any value are loaded as they are; powers of two serve a weight of fp32 scales too."""
    M, N, K = 50, 264, 1088
    A, W, _ = test_fp8.layer(M, N, K, seed=2)
    weight = fp8.quantize(W.cuda())
    other = fp8.Weight(N, K)
    other.storage.view(torch.uint8).fill_(0x7F)
    other.scales.fill_(torch.nan)
    assert other.load(weight.codes, weight.scales) is other
    assert torch.equal(other.storage.view(torch.uint8), weight.storage.view(torch.uint8))
    assert torch.equal(fp8.forward(A.cuda(), other), fp8.forward(A.cuda(), weight))
    scales = torch.rand(weight.scales.shape, generator=torch.Generator().manual_seed(1)) + 0.5
    other.load(weight.codes, scales.cuda())
    s = scales.double().repeat_interleave(128, -2)[:, :K // 8].repeat_interleave(128, -1)[..., :N]
    assert_product(fp8.forward(A.cuda(), other), test_fp8.rounded(A, 1, 128), (weight.codes.double().cpu() * s).numpy(),
                   "rmk,rkn->mn", K)
    powers = fp8.quantize(W.cuda(), scales=E8M0)
    other.load(powers.codes, powers.scales)
    assert torch.equal(other.scales, torch.exp2(powers.scales.view(torch.uint8).float() - 127))
    assert_product(fp8.forward(A.cuda(), other), test_fp8.rounded(A, 1, 128),
                   (powers.codes.float().cpu() * other.scales.cpu().repeat_interleave(128, -2)[:, :K // 8].repeat_interleave(
                       128, -1)[..., :N]).double().numpy(), "rmk,rkn->mn", K)


@pytest.mark.gpu
def test_the_forms_side_by_side():
    """Both forms' calls on one workspace, in turn, give what each gives alone."""
    M, N, K = 200, 264, 1088
    A, W, dY = (t.cuda() for t in test_fp8.layer(M, N, K, seed=4))
    weights = [fp8.quantize(W, scales=s) for s in (F32, E8M0)]
    want = []
    for w in weights:
        ck = fp8.Checkpoint(M, K)
        want.append([fp8.forward(A, w, checkpoint=ck), *fp8.backward(dY, w, ck)])
    assert not torch.equal(want[0][0], want[1][0])
    ws, cks = fp8.new_workspace(M, weights[0]), [fp8.Checkpoint(M, K) for _ in weights]
    for _ in range(2):
        got = [[fp8.forward(A, w, checkpoint=ck, workspace=ws)] for w, ck in zip(weights, cks)]
        for i, (w, ck) in enumerate(zip(weights, cks)):
            got[i] += fp8.backward(dY, w, ck, workspace=ws)
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


SPARSE = [(3, 136, 40960), (5, 1032, 28672), (24, 2056, 8256), (64, 264, 28672), (100, 520, 8256), (256, 264, 28672), (300, 136, 16384),
          (257, 776, 8256), (700, 264, 2624)]


def sparse(M, N, K, seed):
    """Values of -1, 0 and 1 of which few meet: every sum below 257 in magnitude, exact in bf16, whatever its order."""
    g = torch.Generator().manual_seed(seed)

    def pick(*shape, share):
        sign = torch.randint(0, 2, shape, generator=g) * 2 - 1
        return (sign * (torch.rand(shape, generator=g) < share)).to(BF16)

    share = min(1.0, (1024 / K) ** 0.5)
    return pick(8, M, K // 8, share=share), pick(8, K // 8, N, share=share), pick(M, N, share=min(1.0, (256 / max(M, N)) ** 0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("form", [F32, E8M0])
@pytest.mark.parametrize("M,N,K", SPARSE)
def test_sparse_integers_are_exact_at_any_length(M, N, K, form):
    """A step of 128 that is left out, doubled or scaled by another block's scale shows in every output that it reaches.

    With fp32 scales a 1 stands for 448 fp32(1 / 448), off by at most 2**-23, so that a product of two is off by 2**-21
    of it with the roundings of its scaling, and a sum of at most 4096 of them in at most 400 steps by
    4096 * (2**-21 + 400 * 2**-24), less than 0.11: as whole numbers they are equal."""
    A, W, dY = sparse(M, N, K, M + K)
    W[3, 5:9] *= 2  # blocks of other scales
    dY[M // 2:] *= 2
    weight, ck = fp8.quantize(W.cuda(), scales=form), fp8.Checkpoint(M, K)
    out = fp8.forward(A.cuda(), weight, checkpoint=ck)
    dA, dW = fp8.backward(dY.cuda(), weight, ck)
    alone = fp8.backward(dY.cuda(), weight, None, out=(torch.empty_like(dA), None))[0]
    for got, eq, a, b in ((out, "rmk,rkn->mn", A, W), (dA, "mn,rkn->rmk", dY, W), (alone, "mn,rkn->rmk", dY, W),
                          (dW, "rmk,mn->rkn", A, dY)):
        ref = torch.einsum(eq, a.float(), b.float())  # whole numbers below 2**24: exact
        assert ref.abs().max() <= 256 and ref.abs().max() > 4
        assert torch.einsum(eq, a.abs().float(), b.abs().float()).max() <= 4096
        assert torch.equal(whole(got, form), ref)


def whole(got, form):
    got = got.float().cpu()
    return got if form is E8M0 else got.round() + 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("form", [F32, E8M0])
@pytest.mark.parametrize("T,E,k,N,K", [(4, 4, 2, 136, 16384), (40, 8, 3, 264, 8256), (900, 3, 2, 264, 2624), (300, 5, 2, 776, 8256)])
def test_sparse_integers_through_experts(T, E, k, N, K, form):
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    rows, offsets, pairs = test_moe.order(ids, E)
    A, _, dout = sparse(T * k, N, K, T)
    dout = dout[:T].contiguous()
    W = torch.stack([sparse(1, N, K, e)[1] for e in range(E)])
    r, weight = moe.arrange(ids.cuda(), torch.ones(T, k).cuda(), E), fp8.quantize(W.cuda(), scales=form)
    ck = moe.Checkpoint(r, weight)
    out = moe.forward(A.cuda(), weight, r, checkpoint=ck)
    dA, dW, _ = moe.backward(dout.cuda(), weight, r, ck)
    dy = dout.float()[(pairs // k).long()]
    y = torch.zeros(T * k, N)
    for e in range(E):
        i = slice(int(offsets[e]), int(offsets[e + 1]))
        y[i] = torch.einsum("rmk,rkn->mn", A[:, i].float(), W[e].float())
        assert torch.equal(whole(dA[:, i], form), torch.einsum("mn,rkn->rmk", dy[i], W[e].float()))
        assert torch.equal(whole(dW[e], form), torch.einsum("rmk,mn->rkn", A[:, i].float(), dy[i]))
    assert torch.equal(whole(ck.y, form), y)
    assert torch.equal(whole(out, form), y[rows.long()].sum(1))


# ---------------------------------------------------------------- no GPU needed


def test_the_type_of_scales():
    for scales, item in ((None, 4), (F32, 4), (E8M0, 1)):
        weight = fp8.Weight(72, 512, device="cpu", scales=scales)
        assert weight.scales.dtype is (scales or F32) and weight.scales.element_size() == item
    with pytest.raises(ValueError):
        fp8.Weight(72, 512, device="cpu", scales=torch.float16)
    with pytest.raises(ValueError):
        fp8.set_default_scales(torch.uint8)
    try:
        fp8.set_default_scales(E8M0)
        assert fp8.Weight(72, 512, experts=2, device="cpu").scales.dtype is E8M0
    finally:
        fp8.set_default_scales(F32)
    W = torch.zeros(8, 64, 72, dtype=BF16)
    with pytest.raises(ValueError, match="scales are"):
        fp8.quantize(W, out=fp8.Weight(72, 512, device="cpu"), scales=E8M0)


def test_loading_scales():
    codes = torch.zeros(8, 64, 72).to(torch.float8_e4m3fn)
    powers = torch.tensor([0, 1, 120, 127, 128, 254, 255, 3], dtype=torch.uint8).view(8, 1, 1).view(E8M0)
    weight = fp8.Weight(72, 512, device="cpu").load(codes, powers)
    want = torch.tensor([2.0 ** -127, 2.0 ** -126, 2.0 ** -7, 1, 2, 2.0 ** 127, torch.nan, 2.0 ** -124])
    assert torch.equal(weight.scales.flatten().nan_to_num(7.0), want.nan_to_num(7.0))
    with pytest.raises(TypeError):  # fp32 scales are no powers of two
        fp8.Weight(72, 512, device="cpu", scales=E8M0).load(codes, torch.ones(8, 1, 1))
    with pytest.raises(TypeError):
        weight.load(codes, torch.ones(8, 1, 1).double())
    with pytest.raises(ValueError):
        weight.load(codes, torch.ones(8, 1, 2))


def test_a_checkpoint_serves_its_own_form():
    weight, other = (fp8.Weight(72, 512, device="cpu", scales=s) for s in (F32, E8M0))
    ck = fp8.Checkpoint(2, 512, device="cpu")
    ck.scale_type = F32
    with pytest.raises(ValueError, match="written with"):
        fp8.backward(torch.zeros(2, 72, dtype=BF16), other, ck, out=(None, torch.zeros(8, 64, 72, dtype=BF16)), workspace=ck.codes)
    r = moe.Routing(2, 1, 3, device="cpu")
    experts = fp8.Weight(72, 512, experts=3, device="cpu", scales=E8M0)
    ck = moe.Checkpoint(r, experts)
    ck.scale_type = F32
    with pytest.raises(ValueError, match="written with"):
        moe.backward(torch.zeros(2, 72, dtype=BF16), experts, r, ck)


def test_arguments_of_both_forms_are_refused_before_any_cuda_call():
    lib, n = ops_abi.lib(), ctypes.c_size_t()
    sizes = []
    for form in ("", "_e8m0"):
        fn = lambda name: getattr(lib, f"gemm_rs_{name}{form}")  # noqa: E731
        assert fn("fp8_weight_bytes")(0, 64, 512, ctypes.byref(n), None) == G.GEMM_RS_ERR_UNSUPPORTED_SHAPE
        assert fn("fp8_weight_bytes")(3, 264, 2624, None, ctypes.byref(n)) == G.GEMM_RS_OK
        sizes.append(n.value)
        assert fn("fp8_quantize")(1, 64, 512, None, 16, 16, None) == G.GEMM_RS_ERR_INVALID_ARG
        assert fn("fp8_forward")(2, 64, 512, 16, 16, 16, 16, None, 16, 16, None) == G.GEMM_RS_ERR_INVALID_ARG
        assert fn("fp8_backward")(2, 64, 512, 16, 16, None, 16, 16, 16, 16, 16, None) == G.GEMM_RS_ERR_INVALID_ARG
        d = ctypes.byref(ops_abi.gemm_rs_moe_desc(5, 8, 2, 64, 512))
        assert fn("moe_forward")(d, *[16] * 6, None, None, None, 16, None, None) == G.GEMM_RS_ERR_WORKSPACE
        assert fn("moe_backward")(d, *[16] * 13, None, None) == G.GEMM_RS_ERR_WORKSPACE
    assert sizes == [3 * 8 * 3 * 3 * 4, 3 * 8 * 3 * 3]
    # fp32 scales are aligned as every buffer is
    align = G.GEMM_RS_ERR_MISALIGNED
    assert lib.gemm_rs_fp8_quantize(1, 64, 512, 16, 16, 20, None) == align
    assert lib.gemm_rs_fp8_forward(2, 64, 512, 16, 16, 20, None, None, 16, 16, None) == align
    assert lib.gemm_rs_fp8_backward(2, 64, 512, 16, 16, 20, 16, 16, 16, 16, 16, None) == align
    d = ctypes.byref(ops_abi.gemm_rs_moe_desc(5, 8, 2, 64, 512))
    assert lib.gemm_rs_moe_forward(d, 16, 16, 20, 16, 16, 16, None, None, None, 16, 16, None) == align
    assert lib.gemm_rs_moe_backward(d, 16, 16, 20, *[16] * 11, None) == align
