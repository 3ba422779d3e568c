"""A pre-norm residual block with biases, h + W2 gelu(W1 norm(h) + b1) + b2, with 2:4 weights and activations in 8 bits: a few
steps of fine-tuning with AdamW, then decoding one token.

    python examples/mlp_block.py [--tokens 4096] [--width 1024] [--steps 20] [--bits 8]

Bias, GELU and the residual's sum are done where the products' sums are, GELU's input is kept for the backward pass, and one
call of AdamW updates weights, biases and the norm's gain together, its moments in 8 or 32 bits. Master weights are fp32;
the gradients are masked by the 2:4 pattern, so a pruned weight stays at zero.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_sp24_amd as sp  # noqa: E402

BF16 = torch.bfloat16


class SparseLinear:
    """Y = act(X W^T + b) + R with a 2:4 weight in 8 bits; X comes as codes and scales."""

    def __init__(self, out_features, in_features, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.randn(out_features, in_features, generator=g, device="cuda") / (in_features / 2) ** 0.5
        self.weight = sp.sp24_prune_mask(w, keep=2)[1]  # the dense weight with half of it zeroed
        self.bias = torch.zeros(out_features, device="cuda")
        self.code()

    def code(self):
        self.w = sp.sp24_prune_compress_fp8(self.weight)

    def forward(self, codes, scales, activation="none", residual=None):
        self.kept, self.activation = (codes, scales), activation
        y = sp.sp24_gemm_fp8_fused(*self.w, self.bias.numel(), codes, scales, bias=self.bias, activation=activation,
                                   residual=residual, preact=activation != "none")
        y, self.z = y if activation != "none" else (y, None)
        return y

    def backward(self, dy):
        """The input's gradient; those of weight and bias are kept for the step."""
        dz, self.dbias = sp.sp24_epilogue_backward(dy, self.z, self.activation)
        self.dweight = sp.sp24_grad_weight_fp8(dz, *self.kept, meta=self.w[1])
        return dz @ sp.sp24_decompress_fp8(*self.w, *self.weight.shape)


class Block:
    def __init__(self, width, seed=0, bits=8):
        self.gain = torch.ones(width, device="cuda")
        self.gamma = self.gain.to(BF16)
        self.up, self.down = SparseLinear(4 * width, width, seed), SparseLinear(width, 4 * width, seed + 1)
        self.params = [self.up.weight, self.up.bias, self.down.weight, self.down.bias, self.gain]
        self.states = [sp.sp24_adamw_state(p, bits) for p in self.params]
        self.steps = 0

    def forward(self, x):
        codes, scales, self.h, self.rstd = sp.sp24_rmsnorm_fp8(x, self.gamma)
        self.a = self.up.forward(codes, scales, "gelu")
        return self.down.forward(*sp.sp24_quant_fp8(self.a), residual=x)

    def backward(self, dy):
        dx, self.dgamma = sp.sp24_rmsnorm_backward(self.up.backward(self.down.backward(dy)), self.h, self.rstd, self.gamma, dH=dy)
        return dx

    def step(self, rate):
        self.steps += 1
        grads = [self.up.dweight, self.up.dbias, self.down.dweight, self.down.dbias, self.dgamma]
        sp.sp24_adamw(self.params, grads, self.states, self.steps, lr=rate, weight_decay=0.01, seed=1, copies=[None] * 4 + [self.gamma])
        self.up.code()
        self.down.code()


def train(tokens=4096, width=1024, steps=20, rate=1e-3, bits=8):
    """Fits the block to another block's outputs; returns it and the losses."""
    g = torch.Generator(device="cuda").manual_seed(7)
    teacher, block, losses = Block(width, seed=100), Block(width, bits=bits), []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").to(BF16)
        diff = block.forward(x).float() - teacher.forward(x).float()
        losses.append(diff.square().mean())
        block.backward((diff * (2 / diff.numel())).to(BF16))
        block.step(rate)
    return block, [v.item() for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    block, losses = train(a.tokens, a.width, a.steps, bits=a.bits)
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    y = block.forward(torch.randn(1, a.width, device="cuda").to(BF16))
    print(f"one token: output norm {y.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
