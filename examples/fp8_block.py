"""A pre-norm residual block, h + W2 relu(W1 norm(h)), with 2:4 weights and activations in 8 bits: a few steps of
fine-tuning its kept weights, then decoding one token.

    python examples/fp8_block.py [--tokens 4096] [--width 1024] [--steps 20]

What is kept for the backward pass of a Linear is its 8-bit input (codes and scales), a half of bf16; the weight's
gradient reads it as it is. Master weights are fp32; each step prunes and codes them anew, and the gradients are
masked by the 2:4 pattern, so a pruned weight stays at zero.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_sp24_amd as sp  # noqa: E402

BF16 = torch.bfloat16


class SparseLinear:
    """Y = X W^T with a 2:4 weight in 8 bits; X comes as codes and scales."""

    def __init__(self, out_features, in_features, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.randn(out_features, in_features, generator=g, device="cuda") / (in_features / 2) ** 0.5
        self.master = sp.sp24_prune_mask(w, keep=2)[1]  # the dense weight with half of it zeroed
        self.code()

    def code(self):
        self.w = sp.sp24_prune_compress_fp8(self.master)

    def forward(self, codes, scales):
        self.kept = codes, scales
        return sp.sp24_gemm_fp8(*self.w, self.master.shape[0], codes, scales)

    def backward(self, dy):
        """The input's gradient; the weight's is kept for step()."""
        self.grad = sp.sp24_grad_weight_fp8(dy, *self.kept, meta=self.w[1])
        return dy @ sp.sp24_decompress_fp8(*self.w, *self.master.shape)

    def step(self, rate):
        self.master -= rate * self.grad
        self.code()


class Block:
    def __init__(self, width, seed=0):
        self.gamma = torch.ones(width, dtype=BF16, device="cuda")
        self.up, self.down = SparseLinear(4 * width, width, seed), SparseLinear(width, 4 * width, seed + 1)

    def forward(self, x, residual):
        """(the block's output to be added, the residual stream it is to be added to)."""
        codes, scales, self.h, self.rstd = sp.sp24_rmsnorm_fp8(x, self.gamma, residual=residual)
        self.a = torch.relu(self.up.forward(codes, scales))
        return self.down.forward(*sp.sp24_quant_fp8(self.a)), self.h

    def backward(self, dy, dh):
        """Gradient of x and of the residual alike, from those of forward()'s two outputs."""
        da = self.down.backward(dy) * (self.a > 0)
        dx, self.dgamma = sp.sp24_rmsnorm_backward(self.up.backward(da), self.h, self.rstd, self.gamma, dH=dh)
        return dx

    def step(self, rate):
        self.up.step(rate)
        self.down.step(rate)
        self.gamma -= (rate * self.dgamma).to(BF16)


def train(tokens=4096, width=1024, steps=20, rate=0.3):
    """Fits the block to another block's outputs; returns it and the losses."""
    g = torch.Generator(device="cuda").manual_seed(7)
    teacher, block, losses = Block(width, seed=100), Block(width), []
    for _ in range(steps):
        x, r = (torch.randn(tokens, width, generator=g, device="cuda").to(BF16) for _ in range(2))
        want, _ = teacher.forward(x, r)
        y, h = block.forward(x, r)
        diff = y.float() - want.float()
        losses.append(diff.square().mean())
        block.backward((diff * (2 / diff.numel())).to(BF16), torch.zeros_like(h))
        block.step(rate)
    return block, [v.item() for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    block, losses = train(a.tokens, a.width, a.steps)
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    x, r = (torch.randn(1, a.width, device="cuda").to(BF16) for _ in range(2))
    y, h = block.forward(x, r)
    print(f"one token: output norm {y.float().norm().item():.3f}, residual norm {h.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
