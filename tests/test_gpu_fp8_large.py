"""The 8-bit floating-point operators on operands past 4 GiB, where a 32-bit byte or element offset would wrap: the
last rows (and some across the 2 and 4 GiB marks) against the same rows computed alone by the same entry point, which
the small tests compare with the plain forms. Rows do not depend on each other, so equality is bit for bit; the
weight's gradient is compared with the sum of its halves."""
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def rows_of(n):
    """Rows at the start, the end, and around the fractions of n where offsets pass powers of two."""
    some = [0, n // 8, n // 4, n // 2, n - 300]
    return torch.cat([torch.arange(r, r + 300) for r in some]).cuda()


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def randn(*shape, dtype=torch.bfloat16):
    x = torch.empty(*shape, dtype=dtype, device="cuda")
    for part in x.split(1 << 16):
        part.normal_()
    return x


def test_norm_and_back():
    N, K = 330000, 8192  # 5.4 GB a matrix
    say(f"large norm {N}x{K}")
    x, r, g = randn(N, K), randn(N, K), torch.ones(K, dtype=torch.bfloat16, device="cuda")
    at = rows_of(N)
    codes, scales, h, rstd = sp.sp24_rmsnorm_fp8(x, g, residual=r)
    c2, s2, h2, r2 = sp.sp24_rmsnorm_fp8(x[at], g, residual=r[at])
    assert same(codes.view(torch.uint8)[at], c2) and same(scales.view(torch.uint8)[at], s2)
    assert torch.equal(h[at], h2) and torch.equal(rstd[at], r2)
    dx, dg = sp.sp24_rmsnorm_backward(x, h, rstd, g, dH=r)
    assert torch.equal(dx[at], sp.sp24_rmsnorm_backward(x[at], h[at], rstd[at], g, dH=r[at])[0])
    parts = [sp.sp24_rmsnorm_backward(x[i:i + 30000], h[i:i + 30000], rstd[i:i + 30000], g)[1].double() for i in range(0, N, 30000)]
    want = torch.stack(parts).sum(0)
    assert ((dg.double() - want).norm() / want.norm()).item() < 1e-5


def test_many_rows():
    """More rows than one launch takes."""
    N, K = (1 << 20) + 77, 64
    say(f"many rows {N}x{K}")
    x, g = randn(N, K), torch.ones(K, dtype=torch.bfloat16, device="cuda")
    at = torch.cat([torch.arange(0, 100), torch.arange((1 << 20) - 50, N)]).cuda()
    codes, scales, _, rstd = sp.sp24_rmsnorm_fp8(x, g)
    c2, s2, _, r2 = sp.sp24_rmsnorm_fp8(x[at], g)
    assert same(codes.view(torch.uint8)[at], c2) and same(scales.view(torch.uint8)[at], s2) and torch.equal(rstd[at], r2)


def test_quant_gemm_grad():
    N, K, M = 600000, 8192, 272  # codes of 4.9 GB
    say(f"large quant, gemm, grad {N}x{K}")
    codes = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(N, K // 128, dtype=torch.float8_e8m0fnu, device="cuda")
    for i in range(0, N, 100000):
        sp.sp24_quant_fp8(randn(100000, K), codes=codes[i:i + 100000], scales=scales[i:i + 100000])
    at = rows_of(N)
    c, s = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn), scales.view(torch.uint8)[at].view(torch.float8_e8m0fnu)
    w = sp.sp24_prune_compress_fp8(randn(M, K))
    y = sp.sp24_gemm_fp8(*w, M, codes, scales)
    want = c.float() * s.float().repeat_interleave(128, 1) @ sp.sp24_decompress_fp8(*w, M, K, torch.float32).t()
    assert ((y[at].float() - want).norm() / want.norm()).item() < 5e-3
    dy = randn(N, M)
    dw = sp.sp24_grad_weight_fp8(dy, codes, scales)
    parts = [sp.sp24_grad_weight_fp8(dy[i:i + 50000], codes[i:i + 50000], scales[i:i + 50000]).double() for i in range(0, N, 50000)]
    want = torch.stack(parts).sum(0)
    assert ((dw.double() - want).norm() / want.norm()).item() < 1e-5


def test_quant_large_input():
    N, K = 300000, 8192
    say(f"large quant {N}x{K}")
    x = randn(N, K)
    at = rows_of(N)
    codes, scales = sp.sp24_quant_fp8(x)
    c2, s2 = sp.sp24_quant_fp8(x[at])
    assert same(codes.view(torch.uint8)[at], c2) and same(scales.view(torch.uint8)[at], s2)


def test_large_weight():
    M, K = 655400, 16384  # 21 GB dense, 5.4 GB of values, odd row blocks
    say(f"large weight {M}x{K}")
    w = randn(M, K)
    v, m, s = sp.sp24_prune_compress_fp8(w)
    x, xs = sp.sp24_quant_fp8(randn(100, K))
    for n in (3, 100):
        y = sp.sp24_gemm_fp8(v, m, s, M, x[:n], xs[:n])
        for i in (0, M // 256 * 128, (M - 300) // 128 * 128):
            part = sp.sp24_prune_compress_fp8(w[i:min(M, i + 384)])
            rows = min(M, i + 384) - i
            want = x[:n].float() * xs[:n].float().repeat_interleave(128, 1) @ sp.sp24_decompress_fp8(*part, rows, K, torch.float32).t()
            assert ((y[:, i:i + rows].float() - want).norm() / want.norm()).item() < 5e-3
    out = sp.sp24_decompress_fp8(v, m, s, M, K)
    i = (M - 300) // 128 * 128
    part = sp.sp24_prune_compress_fp8(w[i:])
    assert torch.equal(out[i:], sp.sp24_decompress_fp8(*part, M - i, K))
