"""One tensor-parallel block's row-parallel layer, trained and then served with
the operators around it, on one GPU (8 virtual ranks).

Training step (repeated):
  ck = act8.save(A)                the layer's input kept in 8 bits
  y  = sum_r A_r W_r               GEMM + reduce-scatter, one kernel
  r, h = block_norm.forward        norm, gate and residual scale, next norm
  dx, dy, ... = block_norm.backward
  dA, dW = BackwardPlan.run        from dy and the checkpoint
  W, gate and norm weights take a gradient step
Serving: the trained W in 4 bits (w4.quantize, w4.pack), then single tokens
through w4.matvec and block_norm.forward.

  python examples/row_parallel_block.py [--tokens 512] [--hidden 1024] [--inner 4096] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tensor_gemm_reduce_gb300 import act8, block_norm, w4  # noqa: E402
from tensor_gemm_reduce_gb300 import gemm_rs as G  # noqa: E402

BF16 = torch.bfloat16


class Block:
    """y = sum_r A_r W_r, then (r, h) = norms with gate and residual scale."""

    def __init__(self, tokens: int, hidden: int, inner: int, scale: float = 0.5):
        kr = inner // G.WORLD
        self.scale = scale
        self.W = (torch.randn(G.WORLD, kr, hidden, device="cuda") * inner ** -0.5).to(BF16)
        self.w_post = torch.ones(hidden, dtype=BF16, device="cuda")
        self.w_pre = torch.ones(hidden, dtype=BF16, device="cuda")
        self.gate = torch.ones(1, hidden, dtype=BF16, device="cuda")
        # what a training program keeps from step to step
        self.plan = G.Plan(tokens, hidden, inner)
        self.ws = self.plan.new_workspace()
        self.y = torch.empty(tokens, hidden, dtype=BF16, device="cuda")
        self.outputs = block_norm.new_outputs(self.y)
        self.ck = act8.Checkpoint(tokens, inner)
        self.backward_plan = act8.BackwardPlan(tokens, hidden, inner)
        self.backward_ws = self.backward_plan.new_workspace()
        self.norm_grads = block_norm.new_gradients(self.y, self.gate)
        self.norm_ws = block_norm.new_workspace(self.y, self.gate)
        self.dA = torch.empty(self.backward_plan.a_shape, dtype=BF16, device="cuda")
        self.dW = torch.empty_like(self.W)

    def forward(self, A, x):
        act8.save(A, out=self.ck)
        self.plan.run(A, self.W, self.y, self.ws, G.FUSED)
        return block_norm.forward(x, self.y, self.w_post, self.w_pre, gate=self.gate, scale=self.scale,
                                  out=self.outputs)

    def backward(self, dr, dh, x, stats):
        dx, dy, dw_post, dw_pre, dgate = block_norm.backward(
            dr, dh, x, self.y, self.w_post, self.w_pre, stats, gate=self.gate, scale=self.scale,
            out=self.norm_grads, workspace=self.norm_ws)
        self.backward_plan.run(dy, self.W, self.ck, self.dA, self.dW, self.backward_ws)
        return dx, self.dA, (self.dW, dw_post, dw_pre, dgate)

    def parameters(self):
        return self.W, self.w_post, self.w_pre, self.gate


def train(block: Block, A, x, target, steps: int, lr: float):
    """Steps on half the squared error of h, summed; returns the losses."""
    losses = []
    no_dr = torch.zeros_like(x)
    for _ in range(steps):
        _, h, stats = block.forward(A, x)
        error = h - target
        losses.append(0.5 * error.float().square().mean())
        grads = block.backward(no_dr, error / error.shape[0], x, stats)[2]
        for p, g in zip(block.parameters(), grads):
            p.sub_(lr * g)
    for status in (block.plan.status(), block.backward_plan.status()):
        if status != G.GEMM_RS_OK:
            raise RuntimeError(G.strerror(status))
    return [v.item() for v in losses]


def decode(block: Block, A, x, group: int = 128):
    """Each row of A and x as a single token, through 4-bit weights; returns h of all tokens."""
    weight = w4.pack(*w4.quantize(block.W, group), group=group)
    rows = []
    for m in range(x.shape[0]):
        y = w4.matvec(A[:, m:m + 1].contiguous(), weight)
        rows.append(block_norm.forward(x[m:m + 1], y, block.w_post, block.w_pre, gate=block.gate,
                                       scale=block.scale)[1])
    return torch.cat(rows)


def run(tokens=512, hidden=1024, inner=4096, steps=20, lr=0.5, decoded=16):
    torch.manual_seed(0)
    block = Block(tokens, hidden, inner)
    A = torch.randn(G.WORLD, tokens, inner // G.WORLD, device="cuda").to(BF16)
    x = torch.randn(tokens, hidden, device="cuda").to(BF16)
    target = torch.randn(tokens, hidden, device="cuda").to(BF16)
    losses = train(block, A, x, target, steps, lr)
    h = block.forward(A, x)[1][:decoded].float()
    h4 = decode(block, A[:, :decoded].contiguous(), x[:decoded]).float()
    return losses, ((h4 - h).norm() / h.norm()).item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    losses, error = run(a.tokens, a.hidden, a.inner, a.steps, a.lr)
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    print(f"single tokens through 4-bit weights: relative difference {error:.4f}")
