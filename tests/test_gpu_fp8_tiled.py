"""The 8-bit operators' kernels for many tokens and large weights, which the sizes of the other tests hardly reach: the
stages' and scales' rotation, several tiles a workgroup, padded and garbage-filled operands, other streams and graphs.

On 256 compute units the product takes tiles of 256 x 128 or 256 x 256 by the number of tiles, and the weight's gradient
tiles of 256 x 256 or parts of the tokens; each size below names its kernel, and one test checks that it is the one
that runs."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import fp8_ref as ref
from tests.gpu_util import require_gpu, say
from tests.test_gpu_fp8_scales import e8m0, weight

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16

FEW, WIDE128, WIDE256 = "gemm_fp8_fewtok_kernel", "gemm_fp8_tiled_kernel<128", "gemm_fp8_tiled_kernel<256"
ONE, SPLIT, LARGE = "grad_weight_kernel", "add_parts_kernel", "grad_weight_tiled_kernel"
# M, N, the kernel (128 and 256 wide with one tile a workgroup, then with up to two)
PRODUCTS = [(4100, 1000, WIDE128), (8200, 1030, WIDE256), (4100, 4090, WIDE128), (4100, 5770, WIDE256)]
# stages (of 128 columns): 1, 2, 3, 8 (one chunk of scales), 9, 10, 16, 17
COLUMNS = [128, 256, 272, 1024, 1040, 1168, 2048, 2064]
# N, M, K, the kernel
GRADIENTS = [(200, 384, 512, ONE), (2000, 640, 640, SPLIT), (1000, 3608, 3600, LARGE), (70, 3601, 3600, LARGE),
             (65, 4700, 4624, LARGE)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def kernels_of(fn):
    """Names of the kernels that fn launches."""
    fn()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        fn()
        torch.cuda.synchronize()
    names = " ".join(e.key for e in p.key_averages())
    if "kernel" not in names:
        pytest.skip("the profiler shows no kernels here")
    return names


def exact(w, sw, x, sx):
    """Y = X W^T in 64 bits (w, x: numbers without their scales), on the GPU."""
    m, k = w.shape
    rows = np.repeat(2.0 ** (sw.astype(np.float64) - 127), 128, 0)[:m]
    wf = torch.from_numpy(w * np.repeat(rows, 128, 1)[:, :k]).cuda()
    xf = torch.from_numpy(x * np.repeat(2.0 ** (sx.astype(np.float64) - 127), 128, 1)[:, :k]).cuda()
    return xf @ wf.t().contiguous()


def whole(M, N, K, seed=0):
    """Whole numbers with a power of two a block: (w, sw, x, sx); every sum is exact in fp32 and in the instruction."""
    rng = np.random.default_rng(M * 31 + K * 7 + N + seed)
    T = -(-K // 128)
    w = rng.integers(-3, 4, (M, K)).astype(np.float64)
    x = rng.integers(-4, 5, (N, K)).astype(np.float64)
    return w * ref.keep2(w), 127 + rng.integers(-1, 3, (-(-M // 128), T)), x, 127 + rng.integers(-1, 3, (N, T))


def codes_of(x):
    return torch.from_numpy(x).to(torch.float8_e4m3fn).cuda()


def test_sizes_reach_their_kernels():
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are for 256 compute units")
    for M, N, kernel in PRODUCTS + [(300, 40, FEW), (515, 150, FEW)]:
        w, sw, x, sx = whole(M, N, 272)
        v, xc, xs = weight(w, sw), codes_of(x), e8m0(sx)
        names = kernels_of(lambda: sp.sp24_gemm_fp8(*v, M, xc, xs))
        assert kernel in names, (M, N, names)
    for N, M, K, kernel in GRADIENTS:
        dy, (x, xs) = torch.ones(N, (M + 7) // 8 * 8, dtype=BF16, device="cuda")[:, :M], sp.sp24_quant_fp8(torch.ones(N, K, device="cuda"))
        names = kernels_of(lambda: sp.sp24_grad_weight_fp8(dy, x, xs))
        assert kernel in names and (SPLIT in names) == (kernel == SPLIT), (N, M, K, names)


# ---------------------------------------------------------------- the product

@pytest.mark.parametrize("K", COLUMNS)
@pytest.mark.parametrize("M,N,kernel", PRODUCTS)
def test_product_stages(M, N, kernel, K):
    say(f"gemm fp8 stages {M}x{K} N {N}")
    w, sw, x, sx = whole(M, N, K)
    y = sp.sp24_gemm_fp8(*weight(w, sw), M, codes_of(x), e8m0(sx))
    assert torch.equal(y, exact(w, sw, x, sx).to(BF16))


@pytest.mark.parametrize("dtype,extra", [(BF16, 4), (FP16, 5), (BF16, 7), (FP16, 0)])
@pytest.mark.parametrize("M,N,kernel", PRODUCTS)
def test_product_strides_and_garbage(M, N, kernel, dtype, extra):
    """NaN codes behind every row of X, NaN scales behind every row of scales, an output of any pitch, nothing written
    beside it."""
    say(f"gemm fp8 tiled strides {M} N {N} {dtype} {extra}")
    K = 1168
    w, sw, x, sx = whole(M, N, K, 1)
    xd = torch.full((N, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    xd[:, :K] = codes_of(x).view(torch.uint8)
    sd = torch.full((N, sx.shape[1] + 3), 255, dtype=torch.uint8, device="cuda")
    sd[:, :sx.shape[1]] = e8m0(sx).view(torch.uint8)
    y = torch.full((N, M + extra), 7.0, dtype=dtype, device="cuda")
    sp.sp24_gemm_fp8(*weight(w, sw), M, xd.view(torch.float8_e4m3fn)[:, :K], sd.view(torch.float8_e8m0fnu)[:, :sx.shape[1]], out=y[:, :M])
    assert torch.equal(y[:, :M], exact(w, sw, x, sx).to(dtype)) and (y[:, M:] == 7).all()


@pytest.mark.parametrize("M,N,kernel", PRODUCTS)
def test_product_nan(M, N, kernel):
    """NaN scales (first, last and any block) and NaN codes reach their tokens' rows only."""
    say(f"gemm fp8 tiled NaN {M} N {N}")
    w, sw, x, sx = whole(M, N, 1168, 2)
    codes = codes_of(x).view(torch.uint8)
    for n, b in ((0, 0), (130, 9), (131, 4), (N - 1, 8)):
        sx[n, b] = 255
    w[:, 4 * 128:5 * 128 - 124] = 1.0  # every row keeps two of its columns there: a NaN code among all four reaches it
    w[:, 4 * 128 + 2:4 * 128 + 4] = 0.0
    want = exact(w, sw, np.where(sx.repeat(128, 1)[:, :1168] == 255, 0, x), np.where(sx == 255, 127, sx)).to(BF16)
    codes[200, 4 * 128:4 * 128 + 4] = 0x7F
    y = sp.sp24_gemm_fp8(*weight(w, sw), M, codes.view(torch.float8_e4m3fn), e8m0(sx))
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[[0, 130, 131, 200, N - 1]] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("M,N", [(130, 20), (600, 70), (4100, 1000), (8200, 1030)])
def test_product_alignment_error(M, N, dtype):
    """Element by element: in each block every product is off by less than 2^-13 of the block's largest product (not of
    the largest operands'), then T fp32 sums and one rounding."""
    say(f"gemm fp8 alignment {M} N {N} {dtype}")
    K = 1040
    g = torch.Generator().manual_seed(M + N)
    w8 = sp.sp24_prune_compress_fp8((torch.randn(M, K, generator=g) * 0.02).cuda())
    x, xs = sp.sp24_quant_fp8((torch.randn(N, K, generator=g) * torch.randn(K, generator=g).exp()).cuda())
    y = ref.f64(sp.sp24_gemm_fp8(*w8, M, x, xs, out_dtype=dtype))
    at_m, at_n = np.linspace(0, M - 1, 64).astype(int), np.linspace(0, N - 1, 20).astype(int)
    w64 = ref.f64(sp.sp24_decompress_fp8(*w8, M, K, torch.float32))[at_m]
    x64 = ref.values_of(x, xs)[at_n]
    p = ref.blocks((x64[:, None, :] * w64[None, :, :]).reshape(-1, K))
    want, largest, size = p.sum((1, 2)), np.abs(p).max(2).sum(1), np.abs(p).sum((1, 2))
    bound = 1.01 * ref.UNIT[dtype] * np.abs(want) + 64 * 2.0 ** -13 * largest + 20 * ref.U32 * size + 1e-30
    if dtype == FP16:
        bound += 2.0 ** -25  # half the spacing of subnormal outputs
    assert (np.abs(y[np.ix_(at_n, at_m)].reshape(-1) - want) <= bound).all()


# ---------------------------------------------------------------- the weight's gradient

def gradient_case(N, M, K, seed=0):
    g = torch.Generator().manual_seed(N + M + K + seed)
    dy = torch.randn(N, M, generator=g).to(BF16)
    x, xs = sp.sp24_quant_fp8((torch.randn(N, K, generator=g) * torch.randn(K, generator=g).exp()).cuda())
    return dy, x, xs


def behind(t, extra, fill):
    """The same matrix with `extra` bytes of `fill` after every row's end."""
    n, k = t.shape
    buf = torch.full((n, k + extra), fill, dtype=torch.uint8, device="cuda")
    buf[:, :k] = t.view(torch.uint8)
    return buf.view(t.dtype)[:, :k]


@pytest.mark.parametrize("N,M,K,kernel", GRADIENTS)
def test_gradient_strides_nan_and_garbage(N, M, K, kernel):
    """NaN behind the rows of dY, X and the scales is not read; a NaN scale reaches its 128 columns only."""
    say(f"grad weight garbage N {N} {M}x{K}")
    dy, x, xs = gradient_case(N, M, K)
    wide = torch.full((N, M + (-M) % 8 + 24), float("nan"), dtype=BF16, device="cuda")
    wide[:, :M] = dy.cuda()
    plain = torch.zeros(N, M + (-M) % 8, dtype=BF16, device="cuda")
    plain[:, :M] = dy.cuda()
    want = sp.sp24_grad_weight_fp8(plain[:, :M], x, xs)
    dy64, x64 = ref.f64(dy), ref.values_of(x, xs)
    bound = (N + 8) * ref.U32 * (np.abs(dy64).T @ np.abs(x64)) + 1e-30
    assert (np.abs(ref.f64(want) - dy64.T @ x64) <= bound).all()
    xd, sd = behind(x, 48, 0x7F), behind(xs, 3, 255)
    out = torch.full((M, K + 16), 7.0, device="cuda")
    sp.sp24_grad_weight_fp8(wide[:, :M], xd, sd, out=out[:, :K])
    assert torch.equal(out[:, :K], want) and (out[:, K:] == 7).all()
    last = xs.shape[1] - 1
    for n, b in ((0, 1), (N - 1, last)):
        sd[n, b] = torch.tensor(255, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    got = sp.sp24_grad_weight_fp8(wide[:, :M], xd, sd)
    bad = torch.zeros(K, dtype=torch.bool, device="cuda")
    bad[128:256] = True
    bad[128 * last:] = True
    assert torch.isnan(got[:, bad]).all() and torch.equal(got[:, ~bad], want[:, ~bad])


@pytest.mark.parametrize("N,M,K,kernel", GRADIENTS)
def test_gradient_least_and_largest_scales(N, M, K, kernel):
    """Scales 2^-127 and 2^100: products of small whole numbers, exact in fp32 (x times its scale is a bf16 number)."""
    say(f"grad weight scales N {N} {M}x{K}")
    rng = np.random.default_rng(N + M)
    dy, x = rng.integers(-2, 3, (N, M)).astype(np.float64), rng.integers(-4, 5, (N, K)).astype(np.float64)
    T = -(-K // 128)
    sx = np.tile(np.where(np.arange(T) % 2 == 0, 0, 227), (N, 1))
    pad = np.zeros((N, M + (-M) % 8))
    pad[:, :M] = dy
    got = sp.sp24_grad_weight_fp8(torch.from_numpy(pad).to(BF16).cuda()[:, :M], codes_of(x), e8m0(sx))
    want = dy.T @ (x * np.repeat(2.0 ** (sx.astype(np.float64) - 127), 128, 1)[:, :K])
    assert np.array_equal(ref.f64(got), want)


# ---------------------------------------------------------------- streams and graphs

STEPS = [(2000, 640, 640), (1000, 3608, 3600), (1030, 8200, 1040)]  # tokens split, both tiled kernels, 256-wide product


def inputs(seed, N, K, M):
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()  # noqa: E731
    return draw(N, K), draw(N, K), draw(K), sp.sp24_prune_compress_fp8(draw(M, K)), M, draw(N, M)


def step(x, r, gamma, w, M, dy):
    codes, scales, h, rstd = sp.sp24_rmsnorm_fp8(x, gamma, 1e-6, residual=r)
    return (sp.sp24_gemm_fp8(*w, M, codes, scales), sp.sp24_grad_weight_fp8(dy, codes, scales, meta=w[1]),
            *sp.sp24_rmsnorm_backward(x, h, rstd, gamma, dH=r))


@pytest.mark.parametrize("N,M,K", STEPS)
def test_streams_repeat_bit_for_bit(N, M, K):
    say(f"fp8 streams N {N} {M}x{K}")
    ins = [inputs(10 * i, N, K, M) for i in range(3)]
    want = [step(*a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(3):
        got = []
        for s, a in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(step(*a))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


@pytest.mark.parametrize("N,M,K", STEPS)
def test_graph_replays(N, M, K):
    say(f"fp8 graph N {N} {M}x{K}")
    x, r, gamma, w, _, dy = inputs(3, N, K, M)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x, r, gamma, w, M, dy)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, r, gamma, w, M, dy)
    for i in range(4):
        new = inputs(50 + i, N, K, M)
        x.copy_(new[0])
        dy.copy_(new[5])
        want = step(x, r, gamma, w, M, dy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
