"""A stack of residual MLP blocks in 8-bit integers, and the norm's training step.

    python examples/w8a8_mlp.py [--width 1024] [--hidden 4096] [--layers 4] [--tokens 512]

Each block is five calls on the caller's stream:

    h, q, s = norm(x + h)                 tcr_rmsnorm, codes and a scale a token
    gu      = q W_gu^T * s * s_gu         tcr_gemm_i8, gate and up side by side
    q, s    = codes of silu(gate) * up    tcr_quantize_rows_i8
    x       = q W_d^T * s * s_d           tcr_gemm_i8

with the weights quantised once, a scale for each output channel
(tcr_quantize_rows_i8 on the weight matrix).  A prompt runs eagerly, single
tokens as a captured CUDA graph; both are compared with the same blocks in
binary32.  The training step differentiates a norm (tcr_rmsnorm with its rstd,
tcr_rmsnorm_backward) and fits its weight by gradient descent.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import arithmetic_reduction_tensor_gb300 as tcr  # noqa: E402

EPS = 1e-6


class Block:
    """One residual MLP block: float weights, and their codes."""

    def __init__(self, width, hidden, gen):
        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device="cuda") / cols ** 0.5
            return w.to(torch.bfloat16)
        self.norm = (torch.rand(width, generator=gen, device="cuda") + 0.5).to(torch.bfloat16)
        self.gate_up, self.down = weight(2 * hidden, width), weight(width, hidden)
        self.q_gate_up, self.s_gate_up = tcr.tcr_quantize_rows_i8(self.gate_up)
        self.q_down, self.s_down = tcr.tcr_quantize_rows_i8(self.down)
        self.hidden = hidden

    def __call__(self, x, h):
        """(output, residual stream) in bfloat16; h is updated in place."""
        n = tcr.tcr_rmsnorm(x, self.norm, residual=h, eps=EPS, out_dtype=torch.int8, h=h)
        gu = tcr.tcr_gemm_i8(n.y, self.q_gate_up, n.scale, self.s_gate_up)
        q, s = tcr.tcr_quantize_rows_i8(gu[:, self.hidden:], gate=gu[:, :self.hidden])
        return tcr.tcr_gemm_i8(q, self.q_down, s, self.s_down), h

    def reference(self, x, h):
        """The same block in binary32 without codes."""
        h = h + x
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * self.norm.float()
        gu = y @ self.gate_up.float().t()
        g, u = gu[:, :self.hidden], gu[:, self.hidden:]
        return (g * torch.sigmoid(g) * u) @ self.down.float().t(), h


def forward(blocks, x):
    """The stack's output, from bfloat16 embeddings: x + residual at the end."""
    h = torch.zeros_like(x)
    for b in blocks:
        x, h = b(x, h)
    return tcr.tcr_rmsnorm(x, residual=h).y


def reference(blocks, x):
    x = x.float()
    h = torch.zeros_like(x)
    for b in blocks:
        x, h = b.reference(x, h)
    h = h + x
    return h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)


def decoder(blocks, width):
    """(input, output, replay) of the stack for one token, captured once."""
    x = torch.zeros(1, width, dtype=torch.bfloat16, device="cuda")
    forward(blocks, x)                       # loads the kernels
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = forward(blocks, x)
    return x, y, g.replay


def train_norm(width=512, rows=256, steps=60, rate=2.0, seed=0):
    """Losses of gradient descent on a norm's weight towards a target norm."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    goal = torch.rand(width, generator=gen, device="cuda") + 0.5
    weight = torch.ones(width, device="cuda")
    losses = []
    for _ in range(steps):
        x = torch.randn(rows, width, generator=gen, device="cuda")
        r = torch.randn(rows, width, generator=gen, device="cuda")
        o = tcr.tcr_rmsnorm(x, weight, residual=r, eps=EPS, want_rstd=True)
        want = tcr.tcr_rmsnorm(x, goal, residual=r, eps=EPS).y
        diff = o.y - want
        losses.append(diff.square().mean().item())
        _, dweight = tcr.tcr_rmsnorm_backward(diff * (2 / diff.numel()), o.h, weight, o.rstd)
        weight = weight - rate * width / 4 * dweight
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    blocks = [Block(a.width, a.hidden, gen) for _ in range(a.layers)]
    x = torch.randn(a.tokens, a.width, generator=gen, device="cuda").to(torch.bfloat16)
    y, want = forward(blocks, x), reference(blocks, x)
    off = ((y.float() - want).norm() / want.norm()).item()
    print(f"prompt of {a.tokens}: off binary32 by {off:.4f}")
    one, out, step = decoder(blocks, a.width)
    one.copy_(x[:1])
    step()
    print("one token alone equals the prompt's:", torch.equal(out, y[:1]))
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(100):
        step()
    torch.cuda.synchronize()
    print(f"a token through {a.layers} blocks: {(time.perf_counter() - t) * 1e4:.1f} us")
    losses = train_norm()
    print(f"norm's weight fitted: loss {losses[0]:.4f} -> {losses[-1]:.2e}")


if __name__ == "__main__":
    main()
