"""The row-parallel layer for few tokens with 4-bit weights, against the
formula in float64.

Tolerance: code - zero and the inputs are exact in bf16 and their products in
fp32.  A group's sum has at most 128 terms, a rank's share adds at most K/8/32
groups, and 8 shares and 8 parts follow; a tensor core may truncate where it
aligns its addends, so each of these steps is allowed 2 * 2**-24 of the sum of
the absolute terms.  The result is rounded once: half a bf16 step is at most
2**-8 of the value.
"""
import ctypes
import types

import numpy as np
import pytest
import torch

from tensor_gemm_reduce_gb300 import ops_abi, w4
from tensor_gemm_reduce_gb300 import gemm_rs as G

U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def problem(M, N, K, group, zeros, seed=0):
    g = torch.Generator().manual_seed(seed)
    Kr = K // 8
    groups = -(-Kr // group)
    x = torch.randn(8, M, Kr, generator=g)
    x = torch.where(torch.rand(x.shape, generator=g) < 0.05, 8 * x, x).to(torch.bfloat16)
    codes = torch.randint(0, 16, (8, Kr, N), generator=g, dtype=torch.uint8)
    scales = ((0.2 + torch.rand(8, groups, N, generator=g)) * K ** -0.5).to(torch.bfloat16)
    z = torch.randint(0, 16, (8, groups, N), generator=g, dtype=torch.uint8) if zeros else None
    return x, codes, scales, z


def weights(codes, scales, zeros, group):
    Kr = codes.shape[1]
    at = np.arange(Kr) // group
    z = 8.0 if zeros is None else f64(zeros)[:, at]
    return (f64(codes) - z) * f64(scales)[:, at]


def assert_product(out, x, codes, scales, zeros, group):
    w, xv = weights(codes, scales, zeros, group), f64(x)
    ref = np.einsum("rmk,rkn->mn", xv, w)
    mag = np.einsum("rmk,rkn->mn", abs(xv), abs(w))
    steps = 2 * (128 + codes.shape[1] // 32 + 16)
    err = np.abs(f64(out) - ref)
    bound = 2.0 ** -8 * np.abs(ref) + steps * U * mag + 1e-38
    assert (err <= bound).all(), f"worst {np.nanmax(err / bound):.2f} x the bound"


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


# one vector a rank, a ragged cell and group, odd cells, ragged columns, several parts (few columns, long K)
SHAPES = [(1, 8, 64), (1, 16, 512), (3, 136, 576), (8, 128, 1024), (9, 264, 1600), (16, 520, 4160), (5, 1032, 8192),
          (17, 200, 2112), (32, 256, 1536), (1, 128, 28672), (32, 72, 16384), (24, 648, 10304), (1, 2056, 24640)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_matvec_matches_the_formula(M, N, K, group, zeros):
    x, codes, scales, z = problem(M, N, K, group, zeros, seed=M + N + K)
    dx, dc, ds, dz = cuda(x, codes, scales, z)
    weight = w4.pack(dc, ds, dz, group=group)
    ws = w4.new_workspace(weight)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert w4.matvec(dx, weight, out=out, workspace=ws) is out
    assert_product(out, x, codes, scales, z, group)
    for _ in range(3):  # the sums have a fixed order
        assert torch.equal(w4.matvec(dx, weight), out)


# many columns: 4 warps of columns a CTA (up to 16 tokens from 3969 columns on, above from 1985), 8 (above 16 tokens,
# from 3969), with parts of the inner dimension beside them (4104 columns) or not, ragged last columns, and more
# clusters than run at once (from 12288 columns on), where the first weights are not asked for early
WIDE = [(1, 8192, 1024), (3, 4104, 8256), (16, 6152, 1600), (9, 4000, 576), (24, 2568, 1600), (17, 3960, 2112),
        (32, 4104, 2112), (24, 6152, 1088), (4, 12288, 576), (1, 16392, 512), (12, 12296, 1024), (32, 12288, 576)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", WIDE)
@pytest.mark.parametrize("group,zeros", [(128, False), (64, True), (32, True)])
def test_many_columns(M, N, K, group, zeros):
    test_matvec_matches_the_formula(M, N, K, group, zeros)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 4, 7, 8, 10, 15, 16, 23, 25, 31, 32])
def test_every_token_count_gives_the_same_rows(M):
    x, codes, scales, _ = problem(32, 264, 2624, 64, False, seed=6)
    dx, dc, ds = cuda(x, codes, scales)
    weight = w4.pack(dc, ds, group=64)
    assert torch.equal(w4.matvec(dx[:, :M].contiguous(), weight), w4.matvec(dx, weight)[:M])


@pytest.mark.gpu
def test_not_finite_values_stay_in_their_row_and_column():
    x, codes, scales, z = problem(4, 264, 1600, 128, True, seed=2)
    x[3, 1, 77] = float("nan")
    x[5, 2, 0] = float("inf")
    scales[2, 0, 17] = float("nan")
    dx, dc, ds, dz = cuda(x, codes, scales, z)
    out = f64(w4.matvec(dx, w4.pack(dc, ds, dz, group=128)))
    assert np.isnan(out[1]).all() and not np.isfinite(out[2]).any()
    assert np.isnan(out[:, 17]).all()
    assert np.isfinite(out[[0, 3]][:, np.r_[0:17, 18:264]]).all()


@pytest.mark.gpu
def test_high_bits_and_large_zero_points():
    """Only the low four bits of a code count; zero points go up to 127."""
    x, codes, scales, z = problem(2, 72, 640, 32, True, seed=8)
    z = torch.randint(0, 128, z.shape, dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    dx, dc, ds, dz = cuda(x, codes, scales, z)
    out = w4.matvec(dx, w4.pack(dc | 0x50, ds, dz, group=32))
    assert_product(out, x, codes, scales, z, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,group", [(64, 512, 128), (136, 1600, 32), (8, 8256, 64)])
def test_quantize_is_the_defined_rounding(N, K, group):
    g = torch.Generator().manual_seed(N)
    Kr = K // 8
    W = (torch.randn(8, Kr, N, generator=g) * K ** -0.5).to(torch.bfloat16)
    W[1, :group, 3] = 0
    W[2, 5, 4] = float("inf")
    codes, scales = w4.quantize(W.cuda(), group)
    w = W.float().numpy()
    for k in range(0, Kr, group):
        part = w[:, k:k + group]
        top = np.abs(part).max(1)
        with np.errstate(all="ignore"):
            s = torch.from_numpy(top / np.float32(7)).to(torch.bfloat16).float().numpy()
            c = np.clip(np.rint(part / s[:, None]), -8, 7) + 8
        ok = np.isfinite(top)
        c = np.where(np.broadcast_to(ok[:, None] & (s[:, None] > 0), part.shape), c, 8)
        assert np.array_equal(scales[:, k // group].float().cpu().numpy()[ok], s[ok])
        assert scales[:, k // group].isnan().cpu().numpy()[~ok].all()
        assert np.array_equal(codes[:, k:k + group].cpu().numpy(), c.astype(np.uint8))


@pytest.mark.gpu
def test_empty():
    c = torch.zeros(8, 64, 16, dtype=torch.uint8, device="cuda")
    s = torch.ones(8, 1, 16, dtype=torch.bfloat16, device="cuda")
    weight = w4.pack(c, s, group=64)
    assert w4.matvec(torch.zeros(8, 0, 64, dtype=torch.bfloat16, device="cuda"), weight).shape == (0, 16)
    weight = w4.pack(c[:, :0].contiguous(), s[:, :0].contiguous(), group=64)
    out = torch.full((3, 16), 2.0, dtype=torch.bfloat16, device="cuda")
    assert not w4.matvec(torch.zeros(8, 3, 0, dtype=torch.bfloat16, device="cuda"), weight, out=out).any()


@pytest.mark.gpu
def test_tensor_refusals():
    x, codes, scales, z = cuda(*problem(2, 64, 512, 64, True))
    weight = w4.pack(codes, scales, z, group=64)
    with pytest.raises(TypeError):
        w4.matvec(x.float(), weight)
    with pytest.raises(ValueError):
        w4.matvec(x[:, :, :32].contiguous(), weight)
    with pytest.raises(ValueError):
        w4.matvec(x, weight, out=torch.empty(2, 72, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        w4.matvec(x, weight, out=x.view(-1)[:128].view(2, 64))  # the output would overwrite the input
    with pytest.raises(ValueError):
        w4.pack(codes, scales, z, group=32)
    with pytest.raises(TypeError):
        w4.pack(codes, scales.float(), z, group=64)
    with pytest.raises(G.GemmRSError) as e:
        w4.matvec(torch.zeros(8, 33, 64, dtype=torch.bfloat16, device="cuda"), weight)
    assert e.value.code == G.GEMM_RS_ERR_UNSUPPORTED_SHAPE


# ---------------------------------------------------------------- no GPU needed


@pytest.mark.parametrize("M,N,K,group,code", [
    (33, 64, 512, 128, G.GEMM_RS_ERR_UNSUPPORTED_SHAPE), (-1, 64, 512, 128, G.GEMM_RS_ERR_UNSUPPORTED_SHAPE),
    (1, 60, 512, 128, G.GEMM_RS_ERR_UNSUPPORTED_SHAPE), (1, 64, 520, 128, G.GEMM_RS_ERR_UNSUPPORTED_SHAPE),
    (1, 64, 512, 16, G.GEMM_RS_ERR_INVALID_ARG), (1, 64, 512, 0, G.GEMM_RS_ERR_INVALID_ARG),
    (1, (1 << 19) + 8, 512, 128, G.GEMM_RS_ERR_UNSUPPORTED_SHAPE), (1, 64, 512, 128, G.GEMM_RS_ERR_INVALID_ARG),
    (0, 64, 512, 128, G.GEMM_RS_OK)])
def test_refusals_before_any_cuda_call(M, N, K, group, code):
    assert ops_abi.lib().gemm_rs_w4_run(M, N, K, group, 0, None, None, None, None) == code


def test_other_refusals():
    lib = ops_abi.lib()
    n = ctypes.c_size_t()
    assert lib.gemm_rs_w4_bytes(64, 520, 128, 0, ctypes.byref(n)) == G.GEMM_RS_ERR_UNSUPPORTED_SHAPE
    assert lib.gemm_rs_w4_run(1, 64, 512, 128, 0, 24, 16, 16, None) == G.GEMM_RS_ERR_MISALIGNED
    assert lib.gemm_rs_w4_pack(64, 512, 128, None, None, None, None, None) == G.GEMM_RS_ERR_INVALID_ARG
    assert lib.gemm_rs_w4_quantize(64, 512, 128, None, None, None, None) == G.GEMM_RS_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        w4.pack(torch.zeros(8, 64, 8, dtype=torch.uint8), torch.zeros(8, 1, 8, dtype=torch.bfloat16), group=64)


@pytest.mark.parametrize("other", ["scales", "zeros"])
def test_pack_takes_tensors_of_one_device(other):
    """Tensors of two devices, as far as their attributes go."""
    def tensor(shape, dtype, device):
        return types.SimpleNamespace(shape=torch.Size(shape), dtype=dtype, device=torch.device(device), is_cuda=True,
                                     dim=lambda: len(shape), is_contiguous=lambda: True, data_ptr=lambda: 16)

    at = {"codes": "cuda:0", "scales": "cuda:0", "zeros": "cuda:0", other: "cuda:1"}
    with pytest.raises(ValueError, match=f"{other} is on cuda:1"):
        w4.pack(tensor((8, 64, 8), torch.uint8, at["codes"]), tensor((8, 1, 8), torch.bfloat16, at["scales"]),
                tensor((8, 1, 8), torch.uint8, at["zeros"]), group=64)


def test_packed_size_is_near_half_a_byte_a_weight():
    n = ctypes.c_size_t()
    ops_abi.check(ops_abi.lib().gemm_rs_w4_bytes(8192, 8192, 128, 0, ctypes.byref(n)), "")
    assert n.value == 8192 * 8192 // 2 + 2 * 8192 * 8192 // 128
