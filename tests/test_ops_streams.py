"""The operators on a stream that is not the current one: what a call allocates
belongs to the stream that it runs on."""
import contextlib
import types

import pytest
import torch

from tensor_gemm_reduce_gb300 import act8, block_norm, ops_abi, w4

BF16, U8 = torch.bfloat16, torch.uint8


def calls(new, stream):
    """(name, call) of every entry point that allocates; new(dtype, *shape) makes an input."""
    M, D, K, group = 24, 64, 512, 64
    x, y, dr, dh = (new(BF16, M, D) for _ in range(4))
    w_post, w_pre, gate = new(BF16, D), new(BF16, D), new(BF16, 3, D)
    stats = new(torch.float32, 2, M)
    A, W = new(BF16, 8, M, K // 8), new(BF16, 8, K // 8, D)
    codes, scales, zeros = new(U8, 8, K // 8, D), new(BF16, 8, 1, D), new(U8, 8, 1, D)
    ck = types.SimpleNamespace(shape=A.shape, codes=new(U8, 8, M, 128), scales=new(U8, 8, M, 4))
    weight = types.SimpleNamespace(N=D, K=K, group=group, has_zeros=True, data=new(U8, 16))
    return [
        ("norm forward", lambda: block_norm.forward(x, y, w_post, w_pre, gate=gate, stream=stream)),
        ("norm backward", lambda: block_norm.backward(dr, dh, x, y, w_post, w_pre, stats, gate=gate, stream=stream)),
        ("act8 save", lambda: act8.save(A, stream=stream)),
        ("act8 restore", lambda: act8.restore(ck, stream=stream)),
        ("w4 quantize", lambda: w4.quantize(W, group, stream=stream)),
        ("w4 pack", lambda: w4.pack(codes, scales, zeros, group=group, stream=stream)),
        ("w4 matvec", lambda: w4.matvec(A, weight, stream=stream)),
    ]


@pytest.mark.parametrize("given", [True, False])
def test_allocations_belong_to_the_stream(monkeypatch, given):
    """With the library's calls and the allocator's stream replaced: no GPU needed."""
    stream = types.SimpleNamespace(cuda_stream=5, name="given") if given else None
    current, made = ["current"], []

    @contextlib.contextmanager
    def on(s):
        current.append(s.name if s is not None else current[-1])
        yield
        current.pop()

    def recorded(fn):
        def allocate(*args, **kw):
            made.append(current[-1])
            return fn(*args, **kw)
        return allocate

    inputs = calls(lambda dtype, *shape: torch.zeros(shape, dtype=dtype), stream)
    real = ops_abi.lib()
    ok = lambda *a: 0  # noqa: E731
    done = types.SimpleNamespace(norm_forward=ok, norm_backward=ok, act8=ok, w4_matvec=ok)
    host = types.SimpleNamespace(gemm_rs_norm_workspace=real.gemm_rs_norm_workspace, gemm_rs_w4_quantize=ok,
                                 gemm_rs_act8_layout=real.gemm_rs_act8_layout, gemm_rs_w4_pack=ok,
                                 gemm_rs_w4_bytes=real.gemm_rs_w4_bytes)
    monkeypatch.setattr(ops_abi, "ops", lambda: done)
    monkeypatch.setattr(ops_abi, "lib", lambda: host)
    monkeypatch.setattr(ops_abi, "pointer", lambda *a: 16)
    monkeypatch.setattr(ops_abi, "stream_handle", lambda *a: 5)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch, "empty_like", recorded(torch.empty_like))
    for name, call in inputs:
        made.clear()
        call()
        assert made and set(made) == {"given" if given else "current"}, name
        assert current == ["current"], name


@pytest.mark.gpu
def test_memory_of_a_delayed_call_is_not_given_away():
    """The stream is held up while its calls are enqueued; memory of their sizes that the current
    stream allocates and overwrites in the meantime is other memory."""
    torch.manual_seed(4)
    M, D, K = 608, 1024, 4096
    bf16 = lambda *shape: torch.randn(*shape, device="cuda").to(BF16)  # noqa: E731
    x, y, dr, dh = (bf16(M, D) for _ in range(4))
    w_post, w_pre, gate = bf16(D), bf16(D), bf16(4, D)
    A, W, token = bf16(8, M, K // 8), bf16(8, K // 8, D), bf16(8, 3, K // 8)
    stats = block_norm.forward(x, y, w_post, w_pre, gate=gate)[2]

    def results(stream):
        out = list(block_norm.forward(x, y, w_post, w_pre, gate=gate, stream=stream))
        out += block_norm.backward(dr, dh, x, y, w_post, w_pre, stats, gate=gate, stream=stream)
        out.append(act8.restore(act8.save(A, stream=stream), stream=stream))
        codes, scales = w4.quantize(W, 64, stream=stream)
        out.append(w4.matvec(token, w4.pack(codes, scales, group=64, stream=stream), stream=stream))
        return out

    want = results(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        got = results(side)
        sizes = {t.nbytes for t in got} | {block_norm.workspace_bytes(x, gate), 8 * M * K // 8}
        taken = [torch.empty(n, dtype=U8, device="cuda").fill_(0xFF) for n in sizes for _ in range(4)]
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del taken, got
