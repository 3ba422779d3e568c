"""The example's block: its gradients against autograd over the dequantised weights, training that lowers the loss
and keeps the 2:4 pattern, and one decoded token equal to the same token in a batch."""
import importlib.util
import os

import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import fp8_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_block.py")


@pytest.fixture()
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("fp8_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd(example):
    """fp64 autograd over what the backward pass has kept -- the 8-bit inputs of the Linears, the coded weights, the
    stream h -- with the rounding to codes passed straight through. What the block adds to that is the rounding of y, a,
    dy's products and dx to bf16, at most four in a row: within 4 2^-8 by norm."""
    say("example gradients")
    n, width = 256, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, dy = (torch.randn(n, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    block = example.Block(width)
    y, h = block.forward(x, r)
    dx = block.backward(dy, r)
    dense = lambda b: torch.from_numpy(ref.f64(sp.sp24_decompress_fp8(*b.w, *b.master.shape, torch.float32))).requires_grad_()  # noqa: E731
    w1, w2 = dense(block.up), dense(block.down)
    xq, aq = (torch.from_numpy(ref.values_of(*b.kept)) for b in (block.up, block.down))
    hh = h.cpu().double().requires_grad_()
    gamma = torch.ones(width, dtype=torch.float64, requires_grad=True)
    norm = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + 1e-6) * gamma
    through = lambda value, grad_of: value + grad_of - grad_of.detach()  # noqa: E731
    act = (block.a.cpu() > 0).double() * (through(xq, norm) @ w1.t())
    out = through(aq, act) @ w2.t()
    ((out * dy.cpu().double()).sum() + (hh * r.cpu().double()).sum()).backward()

    def near(got, want):
        assert ((got.cpu().double() - want).norm() / want.norm()).item() < 4 * ref.UB

    near(y, out.detach())
    near(dx, hh.grad)
    near(block.dgamma, gamma.grad)
    for b, w in ((block.up, w1), (block.down, w2)):
        kept = torch.from_numpy(ref.keep2(ref.f64(b.master)))
        near(b.grad, w.grad * kept)
        assert (b.grad.cpu()[~kept] == 0).all()


def test_training_lowers_the_loss(example):
    say("example training")
    block, losses = example.train(tokens=512, width=256, steps=12)
    assert losses[-1] < 0.8 * losses[0]
    for b in (block.up, block.down):
        m = b.master.view(b.master.shape[0], -1, 4)
        assert ((m != 0).sum(2) <= 2).all()


def test_one_token_equals_its_batch_row(example):
    say("example one token")
    block = example.Block(512)
    x, r = (torch.randn(8, 512, device="cuda").bfloat16() for _ in range(2))
    y, h = block.forward(x, r)
    y1, h1 = block.forward(x[:1], r[:1])
    assert torch.equal(h[:1], h1)
    assert ((y[:1].float() - y1.float()).norm() / y1.float().norm()).item() < 2.0 ** -7  # another order of fp32 sums, then bf16
