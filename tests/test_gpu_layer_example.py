"""The example's block, which runs the layer operators together: its gradients against autograd over the dequantised weights,
steps that keep the 2:4 pattern, and one decoded token equal to the same token in a batch."""
import importlib.util
import os

import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import fp8_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_block.py")


@pytest.fixture()
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("mlp_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd(example):
    """fp64 autograd over what the backward pass has kept -- the 8-bit inputs of the Linears, the coded weights, GELU's kept
    input -- with the rounding to codes passed straight through. What the block adds to that is the rounding of a, z, dy's
    products, dz and dx to bf16, at most five in a row: within 5 2^-8 by norm."""
    say("mlp example gradients")
    n, width = 256, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(n, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    block = example.Block(width)
    block.up.bias.copy_(torch.randn(4 * width, generator=g, device="cuda") * 0.1)
    block.down.bias.copy_(torch.randn(width, generator=g, device="cuda") * 0.1)
    y = block.forward(x)
    dx = block.backward(dy)
    dense = lambda b: torch.from_numpy(ref.f64(sp.sp24_decompress_fp8(*b.w, *b.weight.shape, torch.float32))).requires_grad_()  # noqa: E731
    w1, w2 = dense(block.up), dense(block.down)
    b1, b2 = (b.bias.cpu().double().requires_grad_() for b in (block.up, block.down))
    xq, aq = (torch.from_numpy(ref.values_of(*b.kept)) for b in (block.up, block.down))
    hh = x.cpu().double().requires_grad_()
    gamma = torch.ones(width, dtype=torch.float64, requires_grad=True)
    norm = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + 1e-6) * gamma
    through = lambda value, grad_of: value + grad_of - grad_of.detach()  # noqa: E731
    z = through(xq, norm) @ w1.t() + b1
    act = z * torch.special.ndtr(z)
    out = through(aq, act) @ w2.t() + b2 + hh
    (out * dy.cpu().double()).sum().backward()

    def near(got, want):
        assert ((got.cpu().double() - want).norm() / want.norm()).item() < 5 * ref.UB

    near(y, out.detach())
    near(block.up.z, z.detach())
    near(dx, hh.grad)
    near(block.dgamma, gamma.grad)
    for b, w, bias in ((block.up, w1, b1), (block.down, w2, b2)):
        kept = torch.from_numpy(ref.keep2(ref.f64(b.weight)))
        near(b.dweight, w.grad * kept)
        near(b.dbias, bias.grad)


@pytest.mark.parametrize("bits", [8, 32])
def test_training_keeps_the_pattern(example, bits):
    say(f"mlp example training, {bits} bits")
    block, losses = example.train(tokens=512, width=256, steps=6, bits=bits)
    assert all(v == v and v < float("inf") for v in losses)
    for b in (block.up, block.down):
        m = b.weight.view(b.weight.shape[0], -1, 4)
        assert ((m != 0).sum(2) <= 2).all()
        assert (b.bias != 0).any()
    assert torch.equal(block.gamma, block.gain.bfloat16()) and (block.gain != 1).any()


def test_one_token_equals_its_batch_row(example):
    say("mlp example one token")
    block = example.Block(512)
    x = torch.randn(8, 512, device="cuda").bfloat16()
    y, y1 = block.forward(x), block.forward(x[:1])
    assert ((y[:1].float() - y1.float()).norm() / y1.float().norm()).item() < 2.0 ** -7  # another order of fp32 sums, then bf16
