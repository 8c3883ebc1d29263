"""The norms around a block with its gate and residual scale, against the
formulas in float64, element by element.

Tolerances.  bf16 outputs are rounded once: half a step is at most 2**-8 of
the value.  Before that the arithmetic is fp32: a row's sums add at most 32
terms in a thread and 10 levels of pairs, each result passes through two such
sums and about ten more roundings, so its error is below 256 * 2**-24 of its
formula with every term taken absolutely ("mag" below); sums over rows add one
rounding for each row and each of the 152 + 8 partial sums.
"""
import ctypes

import numpy as np
import pytest
import torch

from tensor_gemm_reduce_gb300 import block_norm, ops_abi
from tensor_gemm_reduce_gb300 import gemm_rs as G

U = 2.0 ** -24


# ---------------------------------------------------------------- float64 formulas


def reference(x, y, w_post, w_pre, gate, scale, eps):
    M, D = x.shape
    g = np.ones((1, D)) if gate is None else gate
    g = scale * np.repeat(g, M // g.shape[0] if M else 0, axis=0)
    with np.errstate(all="ignore"):
        p = 1 / np.sqrt((y * y).mean(1) + eps)[:, None]
        c = g * (y * p * w_post)
        r = x + c
        q = 1 / np.sqrt((r * r).mean(1) + eps)[:, None]
        return dict(p=p, q=q, g=g, c=c, r=r, h=r * q * w_pre)


def reference_grads(dr, dh, x, y, w_post, w_pre, gate, scale, eps):
    """{name: (value, magnitude)}: magnitude is the same formula over absolute terms."""
    f = reference(x, y, w_post, w_pre, gate, scale, eps)
    M, D = x.shape
    rows = 1 if gate is None else gate.shape[0]
    out = {}

    def grads(dr, dh, r, y, w_post, w_pre, g, q, p, sign):
        yn, rn, a = y * p, r * q, dh * w_pre
        t = dr + q * (a + sign * rn * (a * rn).mean(1, keepdims=True))
        b = g * t * w_post
        return {"dx": t, "dy": p * (b + sign * yn * (b * yn).mean(1, keepdims=True)),
                "dw_post": (g * t * yn).sum(0), "dw_pre": (dh * rn).sum(0),
                "dgate": (scale * t * yn * w_post).reshape(rows, -1, D).sum(1)}

    val = grads(dr, dh, f["r"], y, w_post, w_pre, f["g"], f["q"], f["p"], -1)
    scale = abs(scale)
    # |x| + |c| in place of r: the branch is added with its own error
    mag = grads(abs(dr), abs(dh), abs(x) + abs(f["c"]), abs(y), abs(w_post), abs(w_pre), abs(f["g"]),
                f["q"], f["p"], +1)
    for k in val:
        if k != "dgate" or gate is not None:
            out[k] = (val[k], mag[k])
    return out


def inputs(M, D, gate_rows, seed=0):
    rng = np.random.default_rng(seed)

    def bf16(a):
        return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)

    t = {"x": bf16(rng.standard_normal((M, D)) * (1 + 4 * (rng.random(D) < 0.02))),
         "y": bf16(rng.standard_normal((M, D)) * np.exp(rng.uniform(-3, 3, (M, 1)))),
         "w_post": bf16(1 + 0.1 * rng.standard_normal(D)), "w_pre": bf16(1 + 0.1 * rng.standard_normal(D)),
         "gate": bf16(0.5 + 0.3 * rng.standard_normal((gate_rows, D))) if gate_rows else None,
         "dr": bf16(0.1 * rng.standard_normal((M, D))), "dh": bf16(0.1 * rng.standard_normal((M, D)))}
    return t


def bf16_ones(*shape):
    return torch.ones(*shape, dtype=torch.bfloat16)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def dev(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def assert_close(got, ref, mag, steps, name):
    got, bound = f64(got), 2.0 ** -8 * np.abs(ref) + steps * U * mag + 1e-38
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - ref) / bound):.2f} x the bound")


# rows and columns at the edges: one row, one vector, a ragged last warp, two to four vectors a thread, fewer and
# more rows than chunks, gate rows that divide, straddle and equal the chunks; gate rows of 7 and 8 rows and rows of
# whole 128-byte lines, where the gate's way into the forward kernel changes
SHAPES = [(1, 8, 0), (1, 8, 1), (3, 64, 3), (2, 264, 2), (5, 1000, 1), (1, 8192, 1), (152, 512, 8), (153, 520, 3),
          (304, 768, 4), (610, 256, 5), (700, 128, 350), (1003, 136, 1003), (960, 72, 6), (17, 4104, 0),
          (9, 8200, 3), (6, 12288, 2), (4, 12296, 1), (5, 16384, 5), (6, 16384, 2), (1520, 1032, 10), (2048, 520, 256), (1050, 264, 150),
          (96, 1024, 4), (1200, 1024, 3), (40, 4160, 2), (310, 1088, 10)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,gate_rows", SHAPES)
@pytest.mark.parametrize("scale", [1.0, -0.37])
def test_forward_matches_the_formula(M, D, gate_rows, scale):
    t = inputs(M, D, gate_rows, seed=M + D)
    d = dev(t)
    r, h, stats = block_norm.forward(d["x"], d["y"], d["w_post"], d["w_pre"], gate=d["gate"], scale=scale, eps=1e-6)
    x, y, w_post, w_pre, gate = (f64(t[k]) for k in ("x", "y", "w_post", "w_pre", "gate"))
    f = reference(x, y, w_post, w_pre, gate, scale, 1e-6)
    mag = np.abs(x) + np.abs(f["c"])
    assert_close(r, f["r"], mag, 256, "r")
    assert_close(h, f["h"], mag * f["q"] * np.abs(w_pre), 256, "h")
    np.testing.assert_allclose(f64(stats), np.stack([f["p"][:, 0], f["q"][:, 0]]), rtol=256 * U)


@pytest.mark.gpu
@pytest.mark.parametrize("gate_rows", [0, 1])
def test_forward_of_many_rows(gate_rows):
    """More traffic than L2 holds: some rows against the formula, which is a row's own."""
    M, D, scale = 4100, 8192, 0.6
    gen = torch.Generator("cuda").manual_seed(3)
    x, y = (torch.randn(M, D, device="cuda", generator=gen).bfloat16() for _ in range(2))
    t = inputs(1, D, gate_rows, seed=5)
    d = dev(t)
    r, h, stats = block_norm.forward(x, y, d["w_post"], d["w_pre"], gate=d["gate"], scale=scale, eps=1e-6)
    rows = torch.tensor([0, 1, 151, 152, 303, 304, 2047, 2048, 4095, 4099], device="cuda")
    xs, ys, w_post, w_pre, gate = f64(x[rows]), f64(y[rows]), f64(t["w_post"]), f64(t["w_pre"]), f64(t["gate"])
    f = reference(xs, ys, w_post, w_pre, gate, scale, 1e-6)
    mag = np.abs(xs) + np.abs(f["c"])
    assert_close(r[rows], f["r"], mag, 256, "r")
    assert_close(h[rows], f["h"], mag * f["q"] * np.abs(w_pre), 256, "h")
    np.testing.assert_allclose(f64(stats[:, rows]), np.stack([f["p"][:, 0], f["q"][:, 0]]), rtol=256 * U)


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,gate_rows", SHAPES)
def test_backward_matches_the_formula(M, D, gate_rows):
    t = inputs(M, D, gate_rows, seed=M * 3 + D)
    d = dev(t)
    scale = 0.7
    args = (d["x"], d["y"], d["w_post"], d["w_pre"])
    stats = block_norm.forward(*args, gate=d["gate"], scale=scale)[2]
    out = block_norm.new_gradients(d["x"], d["gate"])
    for o in out:
        if o is not None:
            o.fill_(float("nan"))  # every element is written
    ws = block_norm.new_workspace(d["x"], d["gate"])
    ws.fill_(0xFF)
    got = block_norm.backward(d["dr"], d["dh"], *args, stats, gate=d["gate"], scale=scale, out=out, workspace=ws)
    got = dict(zip(("dx", "dy", "dw_post", "dw_pre", "dgate"), got))
    ref = reference_grads(*(f64(t[k]) for k in ("dr", "dh", "x", "y", "w_post", "w_pre", "gate")), scale, 1e-6)
    for k, (v, mag) in ref.items():
        steps = 256 + (M + 160 if k.startswith(("dw", "dg")) else 0)
        assert_close(got[k], v, mag, steps, k)
    assert (got["dgate"] is None) == (gate_rows == 0)
    again = block_norm.backward(d["dr"], d["dh"], *args, stats, gate=d["gate"], scale=scale)
    for a, b in zip(again, got.values()):
        assert a is None or torch.equal(a, b)  # the sums have a fixed order


# three vectors a thread (4104 to 5632 and 8200 to 12288 columns) with a gate row for each row, where the weights lie
# in shared memory and the ring has five arrays, and with one or some; four vectors a thread with each
LONG = [(40, 4104, 40), (161, 4608, 161), (9, 5632, 9), (305, 8200, 305), (6, 12288, 6), (154, 12288, 154),
        (306, 5632, 3), (160, 9216, 10), (155, 8200, 1), (4, 12296, 4), (160, 12296, 20), (153, 16384, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,gate_rows", LONG)
def test_long_rows(M, D, gate_rows):
    test_forward_matches_the_formula(M, D, gate_rows, 0.6)
    test_backward_matches_the_formula(M, D, gate_rows)


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,gate_rows", [(6, 32, 0), (6, 32, 1), (6, 40, 3), (160, 16, 4), (5, 24, 5)])
def test_backward_matches_differences(M, D, gate_rows):
    """The directional derivative of sum(dr r + dh h), from the float64 formula alone."""
    t = inputs(M, D, gate_rows, seed=7)
    t["y"] = torch.randn(M, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    d = dev(t)
    scale, eps = 0.7, 1e-6
    args = (d["x"], d["y"], d["w_post"], d["w_pre"])
    stats = block_norm.forward(*args, gate=d["gate"], scale=scale, eps=eps)[2]
    got = dict(zip(("x", "y", "w_post", "w_pre", "gate"),
                   block_norm.backward(d["dr"], d["dh"], *args, stats, gate=d["gate"], scale=scale)))
    names = ["x", "y", "w_post", "w_pre"] + (["gate"] if gate_rows else [])
    base = {k: f64(t[k]) for k in ("x", "y", "w_post", "w_pre", "gate")}
    dr, dh = f64(t["dr"]), f64(t["dh"])
    ref = reference_grads(dr, dh, *base.values(), scale, eps)

    def loss(v):
        f = reference(v["x"], v["y"], v["w_post"], v["w_pre"], v["gate"], scale, eps)
        return (dr * f["r"] + dh * f["h"]).sum()

    rng = np.random.default_rng(1)
    for k in names:
        direction = rng.standard_normal(base[k].shape)
        step = 1e-5
        diff = (loss({**base, k: base[k] + step * direction}) - loss({**base, k: base[k] - step * direction})) / (2 * step)
        v, mag = ref["d" + k]
        # half a bf16 step and the fp32 error of every element; differences: 1e-7 of the terms' size
        bound = (np.abs(direction) * (2.0 ** -8 * np.abs(v) + (416 + M) * U * mag)).sum() + 1e-7 * np.abs(direction * mag).sum()
        assert abs(diff - (direction * f64(got[k])).sum()) <= bound, k


@pytest.mark.gpu
@pytest.mark.parametrize("left", [1.0, 0.1, 1e-3])
def test_a_branch_that_cancels_the_residual(left):
    """r is `left` of x: the sum of r^2 keeps its digits, whatever x and the branch are."""
    M, D = 5, 1032
    rng = np.random.default_rng(3)
    t = inputs(M, D, 1, seed=3)
    y = f64(t["y"])
    p = 1 / np.sqrt((y * y).mean(1, keepdims=True) + 1e-6)
    # w_post = gate = 1: the branch is y p; x is its negative, and a little more, in bf16 steps
    t["w_post"], t["gate"] = bf16_ones(D), bf16_ones(1, D)
    x = torch.from_numpy(-y * p * (1 - left) + 1e-4 * rng.standard_normal((M, D))).to(torch.bfloat16)
    d = dev({**t, "x": x})
    r, h, stats = block_norm.forward(d["x"], d["y"], d["w_post"], d["w_pre"], gate=d["gate"])
    f = reference(f64(x), y, f64(t["w_post"]), f64(t["w_pre"]), f64(t["gate"]), 1.0, 1e-6)
    mag = np.abs(f64(x)) + np.abs(f["c"])
    # an error of 256 * 2**-24 of the terms in each r, and so (by the mean) in q
    drift = 256 * U * np.sqrt((mag * mag).mean(1)) * f["q"][:, 0]
    assert (np.abs(f64(stats[1]) / f["q"][:, 0] - 1) <= 2 * drift).all()
    assert_close(r, f["r"], mag, 256, "r")
    assert_close(h, f["h"], (mag * f["q"] + np.abs(f["r"] * f["q"]) * drift[:, None] / (256 * U)) * np.abs(f64(t["w_pre"])) * 2,
                 256, "h")


# (size of y, of the branch's factor, of x, eps): sum c^2 and sum x c overflow before p brings them back, c = factor y;
# p^2 overflows; c^2 is below the smallest number, and it is all there is of r
FAR = [(3e16, 16.0, 1.0, 1e-6), (3e16, -16.0, 0.0, 1e-6), (2e16, 64.0, 30.0, 0.0), (2e-20, 3.0, 1.0, 0.0),
       (1e-18, 1e-6, 0.0, 0.0), (1e-18, 1e-6, 1e-6, 0.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,gate_rows", [(3, 8192, 1), (4, 264, 2), (3, 72, 3), (2, 12288, 0), (16, 1024, 2)])
@pytest.mark.parametrize("size,factor,x_size,eps", FAR)
def test_a_branch_whose_square_leaves_the_range(M, D, gate_rows, size, factor, x_size, eps):
    """r and its root are of ordinary size, y and the terms of sum r^2 are not.  Products below the
    smallest normal number are off by 2**-150 each: 1e-5 of the 4e-40 that a square of y is at least."""
    rng = np.random.default_rng(D)
    t = inputs(M, D, gate_rows, seed=D)
    signs = rng.choice([-1.0, 1.0], (M, D))
    t["y"] = torch.from_numpy(size * signs * rng.uniform(1, 4, (M, D))).to(torch.bfloat16)
    t["x"] = torch.from_numpy(x_size * rng.standard_normal((M, D))).to(torch.bfloat16)
    scale = 0.5 * factor
    if gate_rows:
        t["gate"] = torch.from_numpy(rng.uniform(1.5, 2.5, (gate_rows, D))).to(torch.bfloat16)
    d = dev(t)
    args = (d["x"], d["y"], d["w_post"], d["w_pre"])
    r, h, stats = block_norm.forward(*args, gate=d["gate"], scale=scale, eps=eps)
    host = [f64(t[k]) for k in ("x", "y", "w_post", "w_pre", "gate")]
    f = reference(*host, scale, eps)
    mag = np.abs(host[0]) + np.abs(f["c"])
    assert_close(r, f["r"], mag, 256, "r")
    assert_close(h, f["h"], mag * f["q"] * np.abs(host[3]), 256, "h")
    np.testing.assert_allclose(f64(stats), np.stack([f["p"][:, 0], f["q"][:, 0]]), rtol=256 * U)
    got = block_norm.backward(d["dr"], d["dh"], *args, stats, gate=d["gate"], scale=scale)
    ref = reference_grads(f64(t["dr"]), f64(t["dh"]), *host, scale, eps)
    assert_close(got[0], *ref["dx"], 256, "dx")
    assert_close(got[3], *ref["dw_pre"], 256 + M + 160, "dw_pre")


@pytest.mark.gpu
def test_rows_with_nothing_or_not_finite_stay_alone():
    """A zero row (eps alone in the root), an infinite and a NaN value change their own rows only."""
    M, D = 8, 256
    t = inputs(M, D, 1)
    t["y"][2] = 0
    t["x"][2] = 0
    t["x"][4, 17] = float("inf")
    t["y"][5, 3] = float("nan")
    d = dev(t)
    r, h, stats = block_norm.forward(d["x"], d["y"], d["w_post"], d["w_pre"], gate=d["gate"])
    f = reference(*(f64(t[k]) for k in ("x", "y", "w_post", "w_pre", "gate")), 1.0, 1e-6)
    for m in range(M):
        if m == 2:
            assert not r[m].any() and not h[m].any()
            assert abs(stats[0, m].item() - 1e3) < 1e-2
        elif m == 5:
            assert r[m].isnan().all() and h[m].isnan().all()
        elif m == 4:
            assert r[m, 17] == float("inf") and h[m, 17].isnan()
            assert torch.isfinite(r[m, :17]).all() and not h[m, :17].any()
        else:
            assert_close(r[m], f["r"][m], np.abs(f["r"][m]) + np.abs(f["c"][m]), 256, "r")
    dr = d["dr"].clone()
    dx, dy, *_ = block_norm.backward(dr, d["dh"], d["x"], d["y"], d["w_post"], d["w_pre"], stats, gate=d["gate"])
    for m in (0, 1, 2, 3, 6, 7):
        assert torch.isfinite(dx[m]).all() and torch.isfinite(dy[m]).all()


@pytest.mark.gpu
def test_no_rows():
    t = dev(inputs(0, 64, 0))
    gate = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    for g in (None, gate):
        r, h, stats = block_norm.forward(t["x"], t["y"], t["w_post"], t["w_pre"], gate=g)
        assert r.shape == h.shape == (0, 64)
        out = block_norm.new_gradients(t["x"], g)
        for o in out:
            if o is not None:
                o.fill_(3)
        got = block_norm.backward(t["dr"], t["dh"], t["x"], t["y"], t["w_post"], t["w_pre"], stats, gate=g, out=out)
        assert not got[2].any() and not got[3].any() and (g is None or not got[4].any())


@pytest.mark.gpu
def test_runs_on_the_given_stream():
    t = dev(inputs(300, 1024, 1))
    want = block_norm.forward(t["x"], t["y"], t["w_post"], t["w_pre"], gate=t["gate"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x2 = torch.zeros_like(t["x"])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x2.copy_(t["x"])
    got = block_norm.forward(x2, t["y"], t["w_post"], t["w_pre"], gate=t["gate"], stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_tensor_refusals():
    t = dev(inputs(4, 64, 1))
    args = [t["x"], t["y"], t["w_post"], t["w_pre"]]
    with pytest.raises(TypeError):
        block_norm.forward(t["x"].float(), *args[1:])
    with pytest.raises(ValueError):
        block_norm.forward(t["x"][:, :32], t["y"][:, :32], t["w_post"][:32], t["w_pre"][:32])  # not contiguous
    with pytest.raises(ValueError):
        block_norm.forward(t["x"], t["y"][:3], t["w_post"], t["w_pre"])
    with pytest.raises(ValueError):
        block_norm.forward(*args, gate=torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        block_norm.forward(*args, out=(t["x"], torch.empty_like(t["x"]), torch.empty(2, 4, device="cuda")))
    with pytest.raises(G.GemmRSError) as e:  # one element off a 16-byte boundary
        flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
        block_norm.forward(flat[1:257].view(4, 64), *args[1:])
    assert e.value.code == G.GEMM_RS_ERR_MISALIGNED
    stats = torch.ones(2, 4, device="cuda")
    with pytest.raises(ValueError):
        block_norm.backward(t["dr"], t["dh"], *args, stats, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- no GPU needed


@pytest.mark.parametrize("kw,code", [
    (dict(D=0), G.GEMM_RS_ERR_UNSUPPORTED_SHAPE), (dict(D=12), G.GEMM_RS_ERR_UNSUPPORTED_SHAPE),
    (dict(D=16392), G.GEMM_RS_ERR_UNSUPPORTED_SHAPE), (dict(M=-1), G.GEMM_RS_ERR_UNSUPPORTED_SHAPE),
    (dict(gate_rows=3), G.GEMM_RS_ERR_UNSUPPORTED_SHAPE), (dict(gate_rows=16), G.GEMM_RS_ERR_UNSUPPORTED_SHAPE),
    (dict(gate_rows=-1), G.GEMM_RS_ERR_INVALID_ARG), (dict(eps=-1.0), G.GEMM_RS_ERR_INVALID_ARG),
    (dict(eps=float("nan")), G.GEMM_RS_ERR_INVALID_ARG), (dict(scale=float("inf")), G.GEMM_RS_ERR_INVALID_ARG),
    (dict(), G.GEMM_RS_ERR_INVALID_ARG)])  # null pointers
def test_refusals_before_any_cuda_call(kw, code):
    d = ops_abi.gemm_rs_norm_desc(**{**dict(M=8, D=64, gate_rows=0, scale=1.0, eps=1e-6), **kw})
    assert ops_abi.lib().gemm_rs_norm_forward(ctypes.byref(d), *[None] * 9) == code
    assert ops_abi.lib().gemm_rs_norm_backward(ctypes.byref(d), *[None] * 15) == code
    n = ctypes.c_size_t()
    rc = ops_abi.lib().gemm_rs_norm_workspace(ctypes.byref(d), ctypes.byref(n))
    assert rc == (code if kw else G.GEMM_RS_OK)


def test_workspace_bytes():
    def need(M, D, gate_rows):
        d = ops_abi.gemm_rs_norm_desc(M, D, gate_rows, 1.0, 0.0)
        n = ctypes.c_size_t()
        ops_abi.check(ops_abi.lib().gemm_rs_norm_workspace(ctypes.byref(d), ctypes.byref(n)), "")
        return n.value

    assert need(0, 64, 0) > 0
    assert need(8192, 8192, 1) == need(8192, 8192, 0) <= 152 * 2 * 8192 * 4
    assert need(8192, 8192, 8192) <= 152 * 4 * 8192 * 4  # not a row for each gate row


def test_host_tensors_are_refused():
    t = inputs(4, 64, 0)
    with pytest.raises(ValueError):
        block_norm.forward(t["x"], t["y"], t["w_post"], t["w_pre"])
