"""The example that trains and serves a block with the layer and the operators
around it, against the same steps in float64."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("row_parallel_block",
                                                  os.path.join(ROOT, "examples", "row_parallel_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def layer64(A, x, W, w_post, w_pre, gate, scale):
    y = torch.einsum("rmk,rkn->mn", A, W)
    u = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w_post
    r = x + scale * gate * u
    return r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * w_pre


@pytest.mark.gpu
def test_one_training_step_is_the_layers_gradient(example):
    """Through the whole chain: the 8 bits of A (7 and a sign against the largest of 32
    values of a normal distribution: 1% of its norm), and bf16 at each of five hand-overs
    (2^-9 of a value on average), keep each gradient's direction to 3%."""
    torch.manual_seed(1)
    tokens, hidden, inner = 136, 264, 1600
    block = example.Block(tokens, hidden, inner)
    A = torch.randn(8, tokens, inner // 8, device="cuda").to(torch.bfloat16)
    x = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    dh = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    _, h, stats = block.forward(A, x)
    dx, dA, grads = block.backward(torch.zeros_like(x), dh, x, stats)
    leaves = [t.double().requires_grad_(True) for t in (A, x, *block.parameters())]
    ref_h = layer64(*leaves, block.scale)
    assert (h.double() - ref_h).norm() <= 0.03 * ref_h.norm()
    ref = torch.autograd.grad(ref_h, leaves, dh.double())
    for got, want in zip((dA, dx, *grads), ref):
        assert (got.double() - want).norm() <= 0.03 * want.norm()


@pytest.mark.gpu
def test_training_lowers_the_loss_and_decoding_agrees(example):
    losses, error = example.run(tokens=256, hidden=512, inner=2048, steps=8, decoded=4)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    # 4 bits against a group's largest of 128 normal values: a step of 2.6/7 of the
    # deviation, so 0.11 of the weights' norm, and scale = 0.5 of the branch beside x
    assert error < 0.11
