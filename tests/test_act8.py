"""8-bit checkpoints of the row-parallel layer's input, and its backward pass.

A checkpoint's values are defined exactly, so they are compared bit for bit.

Tolerance of the backward pass: its operands are exact in bf16, products are
exact in fp32, and a sum of n terms in fp32 (in any order, with a tensor core
that may truncate where it aligns its addends) is within 2 n 2**-24 of the sum
of the absolute terms; the result is rounded once to bf16, half a step being at
most 2**-8 of the value.
"""
import ctypes

import numpy as np
import pytest
import torch

from tensor_gemm_reduce_gb300 import act8, ops_abi
from tensor_gemm_reduce_gb300 import gemm_rs as G

U = 2.0 ** -24
BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def checkpoint_values(a):
    """The values a checkpoint of float64 a [8][M][Kr] stands for, by the definition."""
    out = np.empty_like(a)
    for k in range(0, a.shape[-1], act8.GROUP):
        g = a[..., k:k + act8.GROUP]
        top = np.abs(g).max(-1, keepdims=True)
        with np.errstate(all="ignore"):
            e = np.full(top.shape, -126)
            for _ in range(260):
                e = np.where(top > 127 * np.exp2(e.astype(float)), e + 1, e)
            s = np.exp2(e.astype(float))
            v = np.rint(g / s) * s
            v = np.where(np.abs(v) >= 2.0 ** 128, np.sign(v) * 63 * 2.0 ** 122, v)
        out[..., k:k + act8.GROUP] = np.where(np.isfinite(top), v, np.nan)
    return out


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def activations(M, K, seed=0):
    rng = np.random.default_rng(seed)
    a = rng.standard_normal((8, M, K // 8))
    return bf16(np.where(rng.random(a.shape) < 0.05, 8 * a, a))


SHAPES = [(8, 64), (8, 256), (16, 320), (24, 1024), (40, 1088), (128, 1600), (8, 8256), (264, 4096), (1024, 576)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", SHAPES)
def test_checkpoint_is_the_defined_value(M, K):
    A = activations(M, K, seed=M + K)
    ck = act8.Checkpoint(M, K)
    ck.codes.fill_(0xFF)
    ck.scales.fill_(0xFF)
    assert act8.save(A.cuda(), out=ck) is ck
    back = torch.full(ck.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    act8.restore(ck, out=back)
    assert np.array_equal(f64(back), checkpoint_values(f64(A)))
    assert ck.nbytes <= 8 * M * (K // 8 + 128) * 33 / 32


@pytest.mark.gpu
def test_checkpoint_of_every_magnitude():
    """Every finite bf16 value as the largest of its group, with the other values of its size around it."""
    bits = np.arange(0x7F80, dtype=np.int32)
    rng = np.random.default_rng(5)
    rows = []
    for chunk in np.array_split(bits, 8 * 24):
        row = np.zeros(32 * 170, dtype=np.int32)
        for i, b in enumerate(chunk):
            row[32 * i:32 * i + 32] = np.maximum(b - rng.integers(0, 900, 32), 0) | (rng.integers(0, 2, 32) << 15)
            row[32 * i + rng.integers(32)] = b
        rows.append(row)
    a = torch.from_numpy(np.stack(rows).astype(np.uint16).view(np.int16)).view(torch.bfloat16).view(8, 24, 32 * 170)
    back = act8.restore(act8.save(a.cuda()))
    want = checkpoint_values(f64(a))
    assert np.isfinite(f64(back)).all()
    assert np.array_equal(f64(back), want)


@pytest.mark.gpu
def test_groups_that_are_not_finite():
    A = activations(8, 1600, seed=3)  # 200 columns a rank: the last group has 8
    A[0, 0, 3] = float("nan")
    A[1, 2, 40] = float("inf")
    A[7, 7, 199] = float("-inf")
    A[3, 3] = 0
    back = act8.restore(act8.save(A.cuda()))
    want = checkpoint_values(f64(A))
    assert np.array_equal(f64(back), want, equal_nan=True)
    assert np.isnan(want).sum() == 32 + 32 + 8


# ---------------------------------------------------------------- backward pass


def assert_products(dA, dW, dY, W, values):
    dY, W = f64(dY), f64(W)
    M, N = dY.shape
    for got, ref, mag, n in (
            (dA, np.einsum("mn,rkn->rmk", dY, W), np.einsum("mn,rkn->rmk", abs(dY), abs(W)), N),
            (dW, np.einsum("rmk,mn->rkn", values, dY), np.einsum("rmk,mn->rkn", abs(values), abs(dY)), M)):
        if got is None:
            continue
        bound = 2.0 ** -8 * np.abs(ref) + 2 * n * U * mag + 1e-38
        err = np.abs(f64(got) - ref)
        assert (err <= bound).all(), f"worst {np.nanmax(err / bound):.2f} x the bound"


def problem(M, N, K, seed):
    rng = np.random.default_rng(seed)
    A = activations(M, K, seed)
    W = bf16(rng.standard_normal((8, K // 8, N)) * max(K, 1) ** -0.5)
    dY = bf16(rng.standard_normal((M, N)) * 0.05)
    return A, W, dY


def run(M, N, K, A, W, dY, da=True, dw=True, plan=None, ws=None):
    plan = plan or act8.BackwardPlan(M, N, K)
    ws = plan.new_workspace() if ws is None else ws
    nan = float("nan")
    dA = torch.full(plan.a_shape, nan, dtype=torch.bfloat16, device="cuda") if da else None
    dW = torch.full(plan.w_shape, nan, dtype=torch.bfloat16, device="cuda") if dw else None
    plan.run(dY.cuda(), W.cuda() if da else None, act8.save(A.cuda()) if dw else None, dA, dW, ws)
    assert plan.status() == G.GEMM_RS_OK
    return dA, dW


# one token row block, ragged in every dimension, several tiles, single steps, more tiles than pairs
PROBLEMS = [(8, 8, 64), (8, 264, 512), (128, 512, 1024), (392, 776, 1600), (264, 1032, 2112), (72, 2056, 4160),
            (512, 136, 8192), (1040, 520, 576), (256, 4096, 2048), (8, 64, 24576 + 64), (136, 392, 2624), (80, 712, 1216),
            (328, 1144, 448)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", PROBLEMS)
def test_backward_matches_the_formula(M, N, K):
    A, W, dY = problem(M, N, K, seed=M + N + K)
    dA, dW = run(M, N, K, A, W, dY)
    assert_products(dA, dW, dY, W, checkpoint_values(f64(A)))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(392, 776, 1600), (1024, 2048, 4096)])
def test_one_product_alone_and_repeated_runs(M, N, K):
    A, W, dY = problem(M, N, K, seed=9)
    plan = act8.BackwardPlan(M, N, K)
    ws = plan.new_workspace()
    ws.fill_(0xFF)  # an uninitialised workspace
    dA, dW = run(M, N, K, A, W, dY, plan=plan, ws=ws)
    for _ in range(3):
        a, w = run(M, N, K, A, W, dY, plan=plan, ws=ws)
        assert torch.equal(a, dA) and torch.equal(w, dW)
    assert torch.equal(run(M, N, K, A, W, dY, dw=False, plan=plan, ws=ws)[0], dA)
    assert torch.equal(run(M, N, K, A, W, dY, da=False, plan=plan, ws=ws)[1], dW)


@pytest.mark.gpu
def test_backward_matches_differences():
    """The directional derivative of sum(dY out) by W and by A, from the float64 layer alone."""
    M, N, K = 72, 136, 576
    A, W, dY = problem(M, N, K, seed=4)
    dA, dW = run(M, N, K, A, W, dY)
    a, w, g = checkpoint_values(f64(A)), f64(W), f64(dY)
    rng = np.random.default_rng(2)

    def loss(a, w):
        return (g * np.einsum("rmk,rkn->mn", a, w)).sum()

    for got, at, other in ((dA, a, lambda x: loss(x, w)), (dW, w, lambda x: loss(a, x))):
        v = rng.standard_normal(at.shape)
        diff = (other(at + 0.5 * v) - other(at - 0.5 * v))  # the layer is linear in each: no step error
        # half a bf16 step of every element, and 2 * 136 * 2**-24 of terms that are below 8 in sum
        bound = (np.abs(v) * (2.0 ** -8 * np.abs(f64(got)) + 16 * max(M, N) * U)).sum()
        assert abs(diff - (v * f64(got)).sum()) <= bound


@pytest.mark.gpu
def test_not_finite_values_reach_their_gradients_only():
    M, N, K = 136, 264, 1600
    A, W, dY = problem(M, N, K, seed=11)
    A[2, 5, 64] = float("nan")      # its group of 32 columns of rank 2
    dY[7, 9] = float("inf")
    dA, dW = run(M, N, K, A, W, dY)
    dA, dW = f64(dA), f64(dW)
    assert not np.isfinite(dA[:, 7]).any()
    assert np.isfinite(np.delete(dA, 7, axis=1)).all()
    assert np.isnan(dW[2, 64:96]).all()
    assert np.isfinite(np.delete(dW[2], np.r_[64:96], axis=0)[:, np.r_[0:9, 10:N]]).all()
    assert np.isfinite(np.delete(dW, 2, axis=0)[:, :, np.r_[0:9, 10:N]]).all()


@pytest.mark.gpu
def test_empty_contractions():
    def full(shape):
        return torch.full(shape, 3.0, dtype=torch.bfloat16, device="cuda")

    plan = act8.BackwardPlan(0, 64, 512)
    dW = full(plan.w_shape)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ck = act8.save(torch.empty(8, 0, 64, dtype=torch.bfloat16, device="cuda"))
    plan.run(e, full(plan.w_shape), ck, torch.empty(plan.a_shape, dtype=torch.bfloat16, device="cuda"), dW,
             plan.new_workspace())
    assert not dW.any()
    plan = act8.BackwardPlan(64, 0, 512)
    dA = full(plan.a_shape)
    ck = act8.save(full(plan.a_shape))
    plan.run(torch.empty(64, 0, dtype=torch.bfloat16, device="cuda"),
             torch.empty(plan.w_shape, dtype=torch.bfloat16, device="cuda"), ck, dA,
             torch.empty(plan.w_shape, dtype=torch.bfloat16, device="cuda"), plan.new_workspace())
    assert not dA.any()
    assert act8.restore(act8.save(torch.empty(8, 8, 0, dtype=torch.bfloat16, device="cuda"))).numel() == 0


@pytest.mark.gpu
def test_status_is_the_runs_whatever_becomes_of_its_workspace():
    M, N, K = 72, 136, 576
    A, W, dY = (t.cuda() for t in problem(M, N, K, seed=21))
    plan, ck = act8.BackwardPlan(M, N, K), act8.save(A)
    dA, dW = torch.empty_like(A), torch.empty_like(W)

    def filled():
        return plan.new_workspace().fill_(0xFF)

    for outs in ((dA, dW), (dA, None), (None, dW)):
        for _ in range(3):  # a workspace of the call alone; its place, if it is free, holds something else by now
            plan.run(dY, W, ck, *outs, filled())
            others = [filled() for _ in range(4)]
            assert plan.status() == G.GEMM_RS_OK
            assert all((t == 0xFF).all() for t in others)
            del others
    plan.run(dY, W, ck, None, None, filled())  # nothing to compute
    others = [filled() for _ in range(4)]
    assert plan.status() == G.GEMM_RS_OK
    assert all((t == 0xFF).all() for t in others)


@pytest.mark.gpu
def test_plans_share_a_workspace():
    """The larger one's restored activations do not look like the smaller one's failure."""
    sizes = [(8, 264, 512), (392, 776, 1600), (136, 392, 2624)]
    inputs = [problem(*s, seed=31) for s in sizes]
    plans = [act8.BackwardPlan(*s) for s in sizes]
    ws = max((p.new_workspace() for p in plans), key=lambda t: t.numel()).fill_(0xFF)
    for _ in range(2):
        for size, (A, W, dY), plan in zip(sizes, inputs, plans):
            dA, dW = run(*size, A, W, dY, plan=plan, ws=ws)
            assert all(p.status() == G.GEMM_RS_OK for p in plans[:plans.index(plan) + 1])
            assert_products(dA, dW, dY, W, checkpoint_values(f64(A)))


@pytest.mark.gpu
def test_a_plan_first_seen_by_a_graph():
    M, N, K = 72, 136, 576
    A, W, dY = (t.cuda() for t in problem(M, N, K, seed=22))
    plan, ck = act8.BackwardPlan(M, N, K), act8.save(A)
    ws, dA, dW = plan.new_workspace().fill_(0xFF), torch.empty_like(A), torch.empty_like(W)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(dY, W, ck, dA, dW, ws)
    plan.run(dY, W, ck, dA, dW, ws)
    assert plan.status() == G.GEMM_RS_OK
    want = dA.clone(), dW.clone()
    ws.fill_(0xFF)
    dA.zero_()
    dW.zero_()
    graph.replay()
    assert plan.status() == G.GEMM_RS_OK
    assert torch.equal(dA, want[0]) and torch.equal(dW, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(8, 1 << 17, 64), (264, 1 << 16, 2112)])
@pytest.mark.parametrize("da,dw", [(True, True), (True, False)])
def test_a_wait_that_runs_out_is_reported(M, N, K, da, dw):
    """A dA tile's sums take 1024 steps or more, 0.3 ms; the warps that wait for them may wait 1 us.
    The run ends, says so, and leaves nothing behind: the next runs give what the one before gave."""
    A, W, dY = (torch.randn(s, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).to(torch.bfloat16)
                for s in ((8, M, K // 8), (8, K // 8, N), (M, N)))
    ck = act8.save(A)
    good, bad = act8.BackwardPlan(M, N, K), act8.BackwardPlan(M, N, K, timeout_ns=1000)
    ws = good.new_workspace()
    outs = torch.empty_like(A) if da else None, torch.empty_like(W) if dw else None
    good.run(dY, W, ck, *outs, ws)
    assert good.status() == G.GEMM_RS_OK
    want = [None if t is None else t.clone() for t in outs]
    for _ in range(3):
        bad.run(dY, W, ck, *outs, ws)
        assert bad.status() == bad.status() == G.GEMM_RS_ERR_TIMEOUT
        good.run(dY, W, ck, *outs, ws)
        assert good.status() == G.GEMM_RS_OK
        for t, w in zip(outs, want):
            assert t is None or torch.equal(t, w)


@pytest.mark.gpu
def test_tensor_refusals():
    A, W, dY = (t.cuda() for t in problem(16, 64, 512, seed=1))
    with pytest.raises(TypeError):
        act8.save(A.float())
    with pytest.raises(ValueError):
        act8.save(A[:4])
    with pytest.raises(ValueError):
        act8.save(A, out=act8.Checkpoint(24, 512))
    with pytest.raises(ValueError):
        act8.save(A.transpose(0, 1).contiguous().transpose(0, 1))
    plan = act8.BackwardPlan(16, 64, 512)
    ck, ws = act8.save(A), plan.new_workspace()
    dA, dW = torch.empty_like(A), torch.empty_like(W)
    with pytest.raises(ValueError):
        plan.run(dY[:8], W, ck, dA, dW, ws)
    with pytest.raises(ValueError):
        plan.run(dY, W, ck, dA, W, ws)
    with pytest.raises(ValueError):
        plan.run(dY, W, act8.Checkpoint(24, 512), dA, dW, ws)
    with pytest.raises(ValueError):
        plan.run(dY, W, ck, dA, dW, ws[:16])
    plan.run(dY, W, ck, dA, dW, ws)
    assert plan.status() == G.GEMM_RS_OK
    plan.close()
    with pytest.raises(ValueError):
        plan.run(dY, W, ck, dA, dW, ws)


# ---------------------------------------------------------------- no GPU needed


@pytest.mark.parametrize("M,N,K", [(-8, 64, 64), (4, 64, 64), (8, 60, 64), (8, 64, 72), (8, 64, -64),
                                   (1 << 31, 64, 64), (8, 1 << 31, 64), (1 << 28, 64, 1 << 28)])
def test_shapes_are_refused_before_any_cuda_call(M, N, K):
    h, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert (ops_abi.lib().gemm_rs_bwd_create(M, N, K, 0, ctypes.byref(h), ctypes.byref(n))
            == G.GEMM_RS_ERR_UNSUPPORTED_SHAPE)
    assert not h.value


def test_other_refusals():
    lib = ops_abi.lib()
    assert lib.gemm_rs_bwd_create(8, 64, 64, 0, None, None) == G.GEMM_RS_ERR_INVALID_ARG
    assert lib.gemm_rs_bwd_run(*[None] * 9) == G.GEMM_RS_ERR_INVALID_ARG
    assert lib.gemm_rs_bwd_status(None, None) == G.GEMM_RS_ERR_INVALID_ARG
    assert lib.gemm_rs_bwd_destroy(None) == G.GEMM_RS_ERR_INVALID_ARG
    for f in (lib.gemm_rs_act8_save, lib.gemm_rs_act8_restore):
        assert f(8, 64, None, None, None, None) == G.GEMM_RS_ERR_INVALID_ARG
        assert f(4, 64, None, None, None, None) == G.GEMM_RS_ERR_UNSUPPORTED_SHAPE
        assert f(0, 64, None, None, None, None) == G.GEMM_RS_OK
    assert lib.gemm_rs_act8_save(8, 64, 16, 24, 32, None) == G.GEMM_RS_ERR_MISALIGNED
    with pytest.raises(ValueError):
        act8.save(torch.zeros(8, 8, 8, dtype=torch.bfloat16))
