"""The operators inside a CUDA graph: a training step's and a decoding step's
calls, captured once and replayed on new inputs, give what direct calls give."""
import pytest
import torch

from tensor_gemm_reduce_gb300 import act8, block_norm, w4
from tensor_gemm_reduce_gb300 import gemm_rs as G


def bf16(*shape):
    return torch.randn(*shape, device="cuda").to(torch.bfloat16)


@pytest.mark.gpu
def test_a_step_captured_in_a_graph():
    torch.manual_seed(2)
    M, N, K = 136, 520, 1600
    A, W, x, dh, dr = bf16(8, M, K // 8), bf16(8, K // 8, N) * K ** -0.5, bf16(M, N), bf16(M, N), bf16(M, N)
    w_post, w_pre, gate = bf16(N), bf16(N), bf16(4, N)
    token = bf16(8, 1, K // 8)
    plan, back = G.Plan(M, N, K), act8.BackwardPlan(M, N, K)
    ws, back_ws, norm_ws = plan.new_workspace(), back.new_workspace(), block_norm.new_workspace(x, gate)
    weight = w4.pack(*w4.quantize(W, 64), group=64)
    ck, y = act8.Checkpoint(M, K), torch.empty_like(x)
    outs, grads = block_norm.new_outputs(x), block_norm.new_gradients(x, gate)
    dA, dW, out = torch.empty_like(A), torch.empty_like(W), torch.empty(1, N, dtype=torch.bfloat16, device="cuda")

    def step():
        act8.save(A, out=ck)
        plan.run(A, W, y, ws, G.UNFUSED)  # FUSED counts its runs on the host, a replay would not
        stats = block_norm.forward(x, y, w_post, w_pre, gate=gate, out=outs)[2]
        dy = block_norm.backward(dr, dh, x, y, w_post, w_pre, stats, gate=gate, out=grads, workspace=norm_ws)[1]
        back.run(dy, W, ck, dA, dW, back_ws)
        w4.matvec(token, weight, out=out)

    results = lambda: [t.clone() for t in (*outs, *grads, dA, dW, out)]  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (3, 4):
        torch.manual_seed(seed)
        for t in (A, x, dh, dr, token):
            t.copy_(bf16(*t.shape))
        step()
        torch.cuda.synchronize()
        want = results()
        for t in (*outs, *grads, dA, dW, out):
            t.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(results(), want):
            assert torch.equal(a, b)
    assert plan.status() == back.status() == G.GEMM_RS_OK
