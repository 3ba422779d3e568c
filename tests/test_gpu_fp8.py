"""The 8-bit floating-point operators against their plain 64-bit forms (tests/fp8_ref.py).

Tolerances. Codes and scales of given numbers, pruning, decompression and every power-of-two scaling are exact:
compared bit for bit. fp32 sums: n exact products in any order are within n 2^-24 sum|product| of their sum, and a
result in a narrower type is one rounding further (unit roundoff 2^-8 for bf16, 2^-11 for fp16). The norm's mean is a
sum of K squares in chains of at most 32 per thread and then 6 + 16 partial sums, so within 60 2^-24 of itself; its
square root halves that, and the division, the root and the two products add one rounding each: 1 / rms within
36 2^-24, y within 40 2^-24 (NORM below)."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import fp8_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
NORM = 40 * ref.U32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rand(seed, *shape, dtype=torch.float32, spread=0.0):
    """Normal numbers; with spread the columns' sizes vary by exp(spread * normal)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if spread:
        x = x * torch.exp(spread * torch.randn(shape[-1], generator=g))
    return x.to(dtype)


def strided(t: torch.Tensor, extra: int) -> torch.Tensor:
    """The same matrix on the GPU with `extra` more elements (garbage: the type's NaN) between rows."""
    n, k = t.shape
    buf = torch.full((n, k + extra), float("nan"), dtype=torch.float32, device="cuda").to(t.dtype)
    view = buf[:, :k]
    view.copy_(t.cuda())
    return view


def frob(got, want):
    d = np.linalg.norm(got - want)
    return d / max(np.linalg.norm(want), 1e-300)


def make_weight(seed, M, K, score=None):
    """(values, meta, w_scales) on the GPU and the weight they read as (M x K, 64 bits)."""
    w = rand(seed, M, K, dtype=torch.bfloat16) * 0.02
    v, m, s = sp.sp24_prune_compress_fp8(w.cuda())
    w64 = ref.f64(w)
    kept = ref.keep2(w64)
    return (v, m, s), ref.weight(w64, kept), kept


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,K", [(1, 16), (1, 128), (3, 48), (2, 144), (17, 272), (5, 1040), (300, 768), (64, 11008), (3, 40960)])
def test_quant(dtype, N, K):
    say(f"quant {dtype} {N}x{K}")
    x = rand(N + K, N, K, dtype=dtype, spread=2.0)
    codes, scales = sp.sp24_quant_fp8(x.cuda())
    want, e = ref.quant(ref.f64(x))
    assert np.array_equal(ref.f64(codes), want)
    assert np.array_equal(scales.cpu().view(torch.uint8).numpy(), (e + 127).astype(np.uint8))


def test_quant_every_rounding():
    """Every e4m3 number and midpoint, both signs, beside a 448 that fixes the scale at 1."""
    every = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = np.concatenate([every, (every[1:] + every[:-1]) / 2])
    v = np.concatenate([v, -v, np.nextafter(v, 1e9), np.nextafter(v, 0)]).astype(np.float32)
    x = np.full((-(-v.size // 127), 128), 448, np.float32)
    flat = np.full(x.shape[0] * 127, 1.0, np.float32)
    flat[:v.size] = np.clip(v, -448, 448)
    x[:, :127] = flat.reshape(-1, 127)
    codes, scales = sp.sp24_quant_fp8(torch.from_numpy(x).cuda())
    assert (scales.cpu().view(torch.uint8) == 127).all()
    assert np.array_equal(ref.f64(codes), ref.e4m3(x.astype(np.float64)))


@pytest.mark.parametrize("dtype", TYPES)
def test_quant_extremes(dtype):
    info = torch.finfo(dtype)
    tiny = torch.tensor(1, dtype=torch.int16 if info.bits == 16 else torch.int32).view(dtype).item()
    x = torch.zeros(8, 256, dtype=dtype)
    x[1, :128] = info.max
    x[2, 5] = -info.max
    x[3, 7] = tiny
    x[4, :128] = info.tiny
    x[5, 130] = float("inf")
    x[6, 3] = float("nan")
    x[7, 255] = -float("inf")
    x[7, 128] = 1.0
    codes, scales = sp.sp24_quant_fp8(x.cuda())
    byte = scales.cpu().view(torch.uint8).numpy()
    want, e = ref.quant(np.where(np.isfinite(ref.f64(x)), ref.f64(x), 0.0))
    nan = np.zeros_like(byte, bool)
    nan[5, 1] = nan[6, 0] = nan[7, 1] = True
    assert np.array_equal(byte == 255, nan)
    assert np.array_equal(byte[~nan], (e + 127).astype(np.uint8)[~nan])
    ok = np.repeat(~nan, 128, 1)
    assert np.array_equal(ref.f64(codes)[ok], want[ok])


@pytest.mark.parametrize("dtype", TYPES)
def test_quant_strides(dtype):
    N, K = 37, 272
    x = rand(9, N, K, dtype=dtype, spread=1.0)
    codes = torch.zeros(N, K + 32, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros(N, 5, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    sp.sp24_quant_fp8(strided(x, 16), codes=codes[:, :K], scales=scales[:, :3])
    want, e = ref.quant(ref.f64(x))
    assert np.array_equal(ref.f64(codes[:, :K]), want)
    assert np.array_equal(scales.cpu().view(torch.uint8).numpy()[:, :3], (e + 127).astype(np.uint8))
    assert (codes.view(torch.uint8)[:, K:] == 0).all() and (scales.view(torch.uint8)[:, 3:] == 0).all()


# ---------------------------------------------------------------- norm

NORM_SIZES = [(1, 16), (1, 4096), (2, 144), (5, 512), (9, 528), (3, 1024), (7, 1040), (6, 2048), (3, 2064), (5, 4096),
              (3, 4112), (2, 8192), (3, 8208), (2, 16384), (2, 16400), (1, 32768), (197, 768), (1030, 272)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("N,K", NORM_SIZES)
def test_norm(dtype, residual, N, K):
    say(f"norm {dtype} {N}x{K} residual {residual}")
    x, g = rand(N, N, K, dtype=dtype, spread=1.0), (1 + 0.2 * rand(K, K)).to(dtype)
    r = rand(N + 1, N, K, dtype=dtype) if residual else None
    codes, scales, h, rstd = sp.sp24_rmsnorm_fp8(x.cuda(), g.cuda(), 1e-6, residual=None if r is None else r.cuda())
    want_h = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(h.cpu(), want_h)
    y, want_rstd = ref.norm(ref.f64(want_h), ref.f64(g), np.float64(np.float32(1e-6)))
    assert (np.abs(ref.f64(rstd) / want_rstd - 1) <= NORM).all()
    ref.check_codes(codes, scales, y, NORM)


def test_norm_in_place_strides_and_rows():
    """H over X and over the residual, padded rows in every operand, rows of zeros and NaN and infinities."""
    N, K = 41, 784
    for dtype in TYPES:
        x, r = rand(3, N, K, dtype=dtype), rand(4, N, K, dtype=dtype)
        x[2], r[2] = 0, 0
        x[7, 300] = float("nan")
        x[9, 130] = float("inf")
        g = (1 + 0.2 * rand(5, K)).to(dtype)
        want = (x.float() + r.float()).to(dtype)
        for over in ("x", "r"):
            xd, rd = strided(x, 16), strided(r, 48)
            codes, scales, h, rstd = sp.sp24_rmsnorm_fp8(xd, g.cuda(), 1e-5, residual=rd, H=xd if over == "x" else rd)
            assert h.data_ptr() == (xd if over == "x" else rd).data_ptr()
            assert torch.equal(torch.nan_to_num(h.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))
            byte = scales.cpu().view(torch.uint8)
            assert (byte[7] == 255).all()  # a NaN makes its row's mean a NaN
            assert byte[9, 1] == 255 and (ref.f64(codes)[9, :128] == 0).all()  # 1 / rms is 0: inf * 0
            assert (ref.f64(codes)[2] == 0).all() and (byte[2] == 0).all()
            fine = [i for i in range(N) if i not in (7, 9)]
            y, _ = ref.norm(ref.f64(want)[fine], ref.f64(g), np.float64(np.float32(1e-5)))
            ref.check_codes(codes[fine], scales[fine], y, NORM)


def test_norm_zero_row_without_eps():
    _, scales, _, rstd = sp.sp24_rmsnorm_fp8(torch.zeros(1, 128, device="cuda"), torch.ones(128, device="cuda"), 0.0)
    assert torch.isinf(rstd).all() and (scales.view(torch.uint8) == 255).all()


# ---------------------------------------------------------------- gradients of the norm

def back_bounds(dy, h, rstd, gamma, dh, dtype, N, K):
    """Elementwise bounds of dX's and dgamma's errors: the row's mean is a sum of K products (each of three rounded
    products), dX three more roundings of its terms, then the rounding to the type; dgamma a sum of N products."""
    xhat = np.abs(h * rstd[:, None])
    g = np.abs(gamma * dy)
    t = rstd[:, None] * (g + xhat * (g * xhat).mean(1, keepdims=True))
    d = 0 if dh is None else np.abs(dh)
    bx = 70 * ref.U32 * t + 2 * ref.U32 * d + 2 * ref.UNIT[dtype] * (np.abs(t) + d) * (dtype != torch.float32)
    return bx + 1e-30, (N + 4) * ref.U32 * (np.abs(dy) * xhat).sum(0) + 1e-30


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("N,K", NORM_SIZES + [(2500, 512), (9000, 144), (1700, 2064), (600, 8208)])
def test_norm_back(dtype, residual, N, K):
    say(f"norm back {dtype} {N}x{K} dH {residual}")
    h, dy = rand(N, N, K, dtype=dtype, spread=0.5), rand(N + 1, N, K, dtype=dtype)
    g = (1 + 0.2 * rand(K, K)).to(dtype)
    dh = rand(N + 2, N, K, dtype=dtype) if residual else None
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    dx, dg = sp.sp24_rmsnorm_backward(dy.cuda(), h.cuda(), rstd.cuda(), g.cuda(), dH=None if dh is None else dh.cuda())
    a = (ref.f64(dy), ref.f64(h), ref.f64(rstd), ref.f64(g), None if dh is None else ref.f64(dh))
    want_x, want_g = ref.norm_back(*a)
    bx, bg = back_bounds(*a, dtype, N, K)
    assert dx.dtype == dtype and dg.dtype == torch.float32
    assert (np.abs(ref.f64(dx) - want_x) <= bx).all()
    assert (np.abs(ref.f64(dg) - want_g) <= bg).all()


def test_norm_back_against_differences():
    """The gradient of L = sum(dY y(x)) + sum(dH h(x)) by central differences of the plain forward in 64 bits."""
    N, K = 3, 48
    h, dy, dh = (ref.f64(rand(s, N, K)) for s in (1, 2, 3))
    g = 1 + 0.2 * ref.f64(rand(4, K))
    eps = 1e-3
    _, rstd = ref.norm(h, g, eps)

    def loss(hh, gg):
        return (dy * ref.norm(hh, gg, eps)[0]).sum() + (dh * hh).sum()

    f32 = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    dx, dg = sp.sp24_rmsnorm_backward(f32(dy), f32(h), f32(rstd), f32(g), dH=f32(dh))
    for n, k in ((0, 0), (1, 17), (2, 47)):
        d = np.zeros_like(h)
        d[n, k] = 1e-5
        num = (loss(h + d, g) - loss(h - d, g)) / 2e-5
        assert abs(ref.f64(dx)[n, k] - num) <= 1e-5 * (1 + abs(num))
    for k in (0, 31, 47):
        d = np.zeros_like(g)
        d[k] = 1e-5
        num = (loss(h, g + d) - loss(h, g - d)) / 2e-5
        assert abs(ref.f64(dg)[k] - num) <= 1e-5 * (1 + abs(num))


def test_norm_back_in_place_and_strides():
    N, K = 130, 1040
    for dtype in TYPES:
        h, dy, dh = (rand(s, N, K, dtype=dtype) for s in (1, 2, 3))
        g = (1 + 0.2 * rand(4, K)).to(dtype)
        rstd = torch.rsqrt(h.double().square().mean(1)).float()
        first, dg = sp.sp24_rmsnorm_backward(dy.cuda(), h.cuda(), rstd.cuda(), g.cuda(), dH=dh.cuda())
        for over in ("dy", "dh"):
            dyd, dhd = strided(dy, 16), strided(dh, 32)
            out = dyd if over == "dy" else dhd
            again, dg2 = sp.sp24_rmsnorm_backward(dyd, strided(h, 48), rstd.cuda(), g.cuda(), dH=dhd, dX=out)
            assert again.data_ptr() == out.data_ptr() and torch.equal(again, first) and torch.equal(dg, dg2)


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("wanda", [False, True])
@pytest.mark.parametrize("M,K", [(1, 16), (16, 128), (17, 144), (128, 128), (130, 272), (300, 1040), (257, 4096)])
def test_prune_compress_and_back(dtype, wanda, M, K):
    say(f"prune fp8 {dtype} {M}x{K} wanda {wanda}")
    w = rand(M + K, M, K, dtype=dtype, spread=1.0)
    w[:, : K // 2] = (w[:, : K // 2] * 4).round() / 4  # many ties
    norms = torch.rand(K, generator=torch.Generator().manual_seed(K)) if wanda else None
    v, m, s = sp.sp24_prune_compress_fp8(w.cuda(), sp.SP24_SCORE_WANDA if wanda else sp.SP24_SCORE_MAGNITUDE,
                                         norms.cuda() if wanda else None)
    score = w.float().abs().numpy() * (norms.numpy() if wanda else np.float32(1))
    kept = ref.keep2(score)
    want = ref.weight(ref.f64(w), kept)
    assert s.shape == (-(-M // 128), -(-K // 128))
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(ref.f64(sp.sp24_decompress_fp8(v, m, s, M, K, out)), want)
    # the metadata is that of the 2:4 selection of the same type
    if dtype == torch.bfloat16 and not wanda:
        w8 = torch.where(torch.from_numpy(kept), torch.ones(M, K), torch.zeros(M, K)).to(torch.int8)
        assert torch.equal(sp.sp24_prune_compress(w8.cuda())[1], m)
    wide = strided(torch.zeros(M, K), 16)
    sp.sp24_decompress_fp8(v, m, s, M, K, out=wide)
    assert np.array_equal(ref.f64(wide), want)


def test_prune_compress_zero_and_tiny_blocks():
    w = torch.zeros(256, 256)
    w[128, 0], w[0, 200] = 2.0 ** -140, 3e38
    v, m, s = sp.sp24_prune_compress_fp8(w.cuda())
    byte = s.cpu().view(torch.uint8)
    assert byte[0, 0] == 0 and byte[1, 0] == 0 and byte[1, 1] == 0 and byte[0, 1] == 127 + int(ref.scale_exp(np.float64(np.float32(3e38))))
    assert np.array_equal(ref.f64(sp.sp24_decompress_fp8(v, m, s, 256, 256, torch.float32)), ref.weight(ref.f64(w), ref.keep2(ref.f64(w))))


# ---------------------------------------------------------------- the product

GEMM_SIZES = [(1, 16, 1), (16, 128, 1), (17, 144, 2), (130, 272, 3), (257, 128, 16), (300, 1040, 17), (64, 4096, 33),
              (515, 1024, 37), (1100, 272, 64), (129, 2064, 65), (256, 128, 128), (256, 256, 129), (1000, 1152, 200),
              (2050, 400, 300), (4100, 4096, 5), (9000, 256, 40), (18000, 128, 20), (600, 512, 1000), (4096, 640, 513),
              (4100, 272, 4090), (4096, 384, 4096), (8200, 112, 2050), (4100, 144, 1000), (9000, 384, 300), (4100, 128, 900),
              (8200, 256, 4100)]


def int_case(M, K, N, seed=0):
    """Small whole numbers (w in -3..3, x in -4..4) with a power of two for each block: every sum is exact in fp32 and
    in the matrix instruction, so outputs are the rounded 64-bit result bit for bit."""
    rng = np.random.default_rng(M * 31 + K * 7 + N + seed)
    T = -(-K // 128)
    w = rng.integers(-3, 4, (M, K)).astype(np.float64)
    kept = ref.keep2(w)
    w = w * kept
    x = rng.integers(-4, 5, (N, K)).astype(np.float64)
    sx, sw = rng.integers(-1, 3, (N, T)), rng.integers(-1, 3, (-(-M // 128), T))
    v, m, s = sp.sp24_prune_compress_fp8(torch.from_numpy(w).float().cuda())
    # the compressor's own scales make codes of up to 448 units: codes of w and x themselves have the scale 1
    v = (v.float() * s.float().repeat_interleave(8, 0)[:-(-M // 16)].unsqueeze(2).expand(-1, -1, 1024).reshape(-1)).to(torch.float8_e4m3fn)
    as_scale = lambda e: torch.from_numpy((e + 127).astype(np.uint8)).cuda().view(torch.float8_e8m0fnu)  # noqa: E731
    codes = torch.from_numpy(x).to(torch.float8_e4m3fn).cuda()
    x = x * np.repeat(2.0 ** sx, 128, 1)[:, :K]
    w = w * np.repeat(np.repeat(2.0 ** sw, 128, 0)[:M], 128, 1)[:, :K]
    return (v, m, as_scale(sw)), codes, as_scale(sx), x @ w.T


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K,N", GEMM_SIZES)
def test_gemm_whole_numbers(M, K, N, dtype):
    say(f"gemm fp8 whole numbers {M}x{K} N {N} {dtype}")
    w, x, xs, want = int_case(M, K, N)
    y = sp.sp24_gemm_fp8(*w, M, x, xs, out_dtype=dtype)
    assert y.dtype == dtype and torch.equal(y.cpu(), torch.from_numpy(want).to(dtype))


def gemm_case(M, K, N, seed=0):
    w, w64, _ = make_weight(M + K + seed, M, K)
    x, xs = sp.sp24_quant_fp8(rand(N + K + seed, N, K, spread=1.0).cuda())
    x64 = ref.values_of(x, xs)
    return w, x, xs, x64 @ w64.T, x64, w64


def gemm_bound(x64, w64, want, unit):
    """64 products a block, each off by less than 2^-13 of the block's largest (bounded by the operands' largest),
    fp32 sums over the blocks, one rounding to the type."""
    T = -(-x64.shape[1] // 128)
    big = lambda a: np.abs(ref.blocks(a)).max(2)  # noqa: E731
    align = 64 * 2.0 ** -13 * big(x64) @ big(w64).T
    return 1.01 * unit * np.abs(want) + align + (T + 8) * ref.U32 * (np.abs(x64) @ np.abs(w64).T) + 1e-30


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K,N", GEMM_SIZES)
def test_gemm(M, K, N, dtype):
    say(f"gemm fp8 {M}x{K} N {N} {dtype}")
    w, x, xs, want, x64, w64 = gemm_case(M, K, N)
    got = ref.f64(sp.sp24_gemm_fp8(*w, M, x, xs, out_dtype=dtype))
    assert (np.abs(got - want) <= gemm_bound(x64, w64, want, ref.UNIT[dtype])).all()
    # by norm: the rounding, and 64 independent alignment errors of at most 2^-13 of a product (a product's size is
    # the result's over sqrt(32 T) or more, the largest one within 30 of it)
    assert frob(got, want) <= ref.UNIT[dtype] + 30 * 2.0 ** -13 / np.sqrt(32)


@pytest.mark.parametrize("M,K,N", [(130, 272, 1), (130, 272, 20), (300, 400, 70), (515, 528, 257)])
def test_gemm_strides_and_garbage(M, K, N):
    """Padded rows of NaN codes behind X and its scales, an output of any pitch, nothing written beside it."""
    say(f"gemm fp8 strides {M}x{K} N {N}")
    w, x, xs, want = int_case(M, K, N, 5)
    xd = torch.full((N, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    xd[:, :K] = x.view(torch.uint8)
    sd = torch.full((N, xs.shape[1] + 3), 255, dtype=torch.uint8, device="cuda")
    sd[:, :xs.shape[1]] = xs.view(torch.uint8)
    for dtype in (torch.float16, torch.bfloat16):
        for extra in (5, 8):
            y = torch.full((N, M + extra), 7.0, dtype=dtype, device="cuda")
            sp.sp24_gemm_fp8(*w, M, xd.view(torch.float8_e4m3fn)[:, :K], sd.view(torch.float8_e8m0fnu)[:, :xs.shape[1]], out=y[:, :M])
            assert torch.equal(y[:, :M].cpu(), torch.from_numpy(want).to(dtype)) and (y[:, M:] == 7).all()


@pytest.mark.parametrize("N", [3, 40, 150])
def test_gemm_nan_and_scale_range(N):
    """A NaN scale makes its token's row NaN and no other; scales far apart, zero blocks, the smallest scale."""
    say(f"gemm fp8 scales N {N}")
    M, K = 160, 640
    w, x, xs, _, _, w64 = gemm_case(M, K, N, 9)
    byte = xs.view(torch.uint8).clone()
    byte[1, 3] = 255
    byte[0, 0], byte[0, 1], byte[2, 4] = 190, 20, 0
    x64 = ref.f64(x) * np.repeat(2.0 ** (byte.cpu().numpy().astype(np.float64) - 127), 128, 1)
    x64[1] = 0
    want = x64 @ w64.T
    got = ref.f64(sp.sp24_gemm_fp8(*w, M, x, byte.view(torch.float8_e8m0fnu)))
    assert np.isnan(got[1]).all()
    rest = [i for i in range(N) if i != 1]
    assert (np.abs(got - want) <= gemm_bound(x64, w64, want, ref.UB))[rest].all()
    zero = torch.zeros_like(byte).view(torch.float8_e8m0fnu)  # all scales 2^-127
    x64 = ref.f64(x) * 2.0 ** -127
    want = x64 @ w64.T
    got = ref.f64(sp.sp24_gemm_fp8(*w, M, x, zero))
    assert (np.abs(got - want) <= gemm_bound(x64, w64, want, ref.UB) + K * 2.0 ** -133).all()


@pytest.mark.parametrize("N", [2, 11, 16, 25, 43, 64, 130])
@pytest.mark.parametrize("M", [2100, 4100, 6000, 8170, 10000, 12200])
def test_gemm_row_blocks(M, N):
    """One to three row blocks a workgroup, and three that may lie in two rows of weight scales."""
    say(f"gemm fp8 row blocks {M} N {N}")
    w, x, xs, want = int_case(M, 272, N, 3)
    y = sp.sp24_gemm_fp8(*w, M, x, xs)
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_gemm_counts_kept_weights():
    """Ones everywhere: Y counts the kept weights, whatever the tiling (exact)."""
    for M, K, N in ((48, 400, 5), (300, 144, 90), (260, 1040, 260)):
        w = sp.sp24_prune_compress_fp8(torch.ones(M, K, device="cuda"))
        x, xs = sp.sp24_quant_fp8(torch.ones(N, K, device="cuda"))
        assert (sp.sp24_gemm_fp8(*w, M, x, xs, out_dtype=torch.float16) == K / 2).all()


# ---------------------------------------------------------------- the weight's gradient

GRAD_SIZES = [(1, 1, 16), (2, 17, 128), (31, 128, 144), (32, 130, 272), (33, 8, 48), (65, 300, 400), (300, 257, 640),
              (2000, 130, 144), (6304, 136, 256), (1000, 768, 768), (64, 4100, 528), (513, 1024, 2064),
              (1, 4096, 4096), (70, 3601, 3600), (129, 4104, 3856), (700, 3330, 4112)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("N,M,K", GRAD_SIZES)
def test_grad_weight(N, M, K, masked):
    say(f"grad weight N {N} {M}x{K} masked {masked}")
    dy = rand(N + M, N, M, dtype=torch.bfloat16)
    x, xs = sp.sp24_quant_fp8(rand(N + K, N, K, spread=1.0).cuda())
    x64, dy64 = ref.values_of(x, xs), ref.f64(dy)
    want, bound = dy64.T @ x64, (N + 8) * ref.U32 * (np.abs(dy64).T @ np.abs(x64)) + 1e-30
    meta = None
    if masked:
        _, meta, _ = sp.sp24_prune_compress_fp8(rand(M, M, K).cuda())
        kept = ref.keep2(ref.f64(rand(M, M, K)))
        want, bound = want * kept, bound * kept
    dyd = strided(dy, (-M) % 8 + 8)
    dw = sp.sp24_grad_weight_fp8(dyd, x, xs, meta=meta)
    assert dw.dtype == torch.float32 and (np.abs(ref.f64(dw) - want) <= bound).all()
    db = sp.sp24_grad_weight_fp8(dyd, x, xs, meta=meta, out_dtype=torch.bfloat16)
    assert torch.equal(db.cpu(), dw.to(torch.bfloat16).cpu())
    wide = torch.full((M, K + 16), 7.0, device="cuda")
    sp.sp24_grad_weight_fp8(dyd, x, xs, meta=meta, out=wide[:, :K])
    assert torch.equal(wide[:, :K], dw) and (wide[:, K:] == 7).all()


def test_grad_weight_against_differences():
    """L = sum(dY * (X W^T)) is linear in W: its differences are dW."""
    N, M, K = 40, 24, 144
    dy = rand(1, N, M, dtype=torch.bfloat16)
    x, xs = sp.sp24_quant_fp8(rand(2, N, K).cuda())
    dw = ref.f64(sp.sp24_grad_weight_fp8(dy.cuda(), x, xs))
    x64, dy64, w = ref.values_of(x, xs), ref.f64(dy), ref.f64(rand(3, M, K))
    for m, k in ((0, 0), (23, 143), (5, 100)):
        d = np.zeros((M, K))
        d[m, k] = 0.5
        num = (dy64 * (x64 @ (w + d).T)).sum() - (dy64 * (x64 @ (w - d).T)).sum()
        assert abs(dw[m, k] - num) <= 1e-5 * (1 + abs(num))


def test_grad_weight_nan_scale_and_garbage():
    """A NaN scale reaches its block of columns only; NaN codes behind a row are not read."""
    N, M, K = 70, 40, 272
    dy = rand(1, N, M, dtype=torch.bfloat16)
    x, xs = sp.sp24_quant_fp8(rand(2, N, K).cuda())
    want = sp.sp24_grad_weight_fp8(dy.cuda(), x, xs)
    xd = torch.full((N, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    xd[:, :K] = x.view(torch.uint8)
    byte = xs.view(torch.uint8).clone()
    xd = xd.view(torch.float8_e4m3fn)[:, :K]
    assert torch.equal(sp.sp24_grad_weight_fp8(strided(dy, 24), xd, xs), want)
    byte[69, 1] = 255
    got = sp.sp24_grad_weight_fp8(dy.cuda(), xd, byte.view(torch.float8_e8m0fnu))
    assert torch.isnan(got[:, 128:256]).all()
    assert torch.equal(got[:, :128], want[:, :128]) and torch.equal(got[:, 256:], want[:, 256:])


# ---------------------------------------------------------------- streams, graphs, refusals

def block(x, r, g, w, M, dy):
    codes, scales, h, rstd = sp.sp24_rmsnorm_fp8(x, g, 1e-6, residual=r)
    y = sp.sp24_gemm_fp8(*w, M, codes, scales)
    dw = sp.sp24_grad_weight_fp8(dy, codes, scales, meta=w[1])
    dc = torch.matmul(dy, sp.sp24_decompress_fp8(*w, M, x.shape[1]))
    dx, dg = sp.sp24_rmsnorm_backward(dc, h, rstd, g, dH=r)
    return y, dw, dx, dg


def block_inputs(seed, N=200, K=512, M=384):
    w, _, _ = make_weight(seed, M, K)
    bf = torch.bfloat16
    return (rand(seed, N, K, dtype=bf).cuda(), rand(seed + 1, N, K, dtype=bf).cuda(), rand(seed + 2, K, dtype=bf).cuda(), w, M,
            rand(seed + 3, N, M, dtype=bf).cuda())


def test_streams_repeat_bit_for_bit():
    ins = [block_inputs(10 * i) for i in range(3)]
    want = [block(*a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(3):
        got = []
        for s, a in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(block(*a))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_graph_replays():
    """Norm, product and both gradients in one captured graph, replayed over new inputs."""
    x, r, g, w, M, dy = block_inputs(3)

    def ours():
        codes, scales, h, rstd = sp.sp24_rmsnorm_fp8(x, g, 1e-6, residual=r)
        return (sp.sp24_gemm_fp8(*w, M, codes, scales), sp.sp24_grad_weight_fp8(dy, codes, scales, meta=w[1]),
                *sp.sp24_rmsnorm_backward(x, h, rstd, g, dH=r))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ours()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ours()
    for i in range(4):
        x.copy_(rand(50 + i, *x.shape, dtype=torch.bfloat16))
        dy.copy_(rand(60 + i, *dy.shape, dtype=torch.bfloat16))
        want = ours()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    codes, scales = sp.sp24_quant_fp8(x)
    w = sp.sp24_prune_compress_fp8(torch.ones(8, 64, device="cuda"))
    dy = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    for call in (
            lambda: sp.sp24_quant_fp8(x.to(torch.int8)), lambda: sp.sp24_quant_fp8(x.t()), lambda: sp.sp24_quant_fp8(x[0]),
            lambda: sp.sp24_quant_fp8(x, codes=codes[:2]), lambda: sp.sp24_rmsnorm_fp8(x, g.float()),
            lambda: sp.sp24_rmsnorm_fp8(x, g[:32]), lambda: sp.sp24_rmsnorm_fp8(x, g, residual=x.float()),
            lambda: sp.sp24_rmsnorm_fp8(x, g, H=x), lambda: sp.sp24_rmsnorm_backward(x, x, torch.ones(3, device="cuda"), g),
            lambda: sp.sp24_gemm_fp8(*w, 8, x, scales), lambda: sp.sp24_gemm_fp8(*w, 8, codes, scales.view(torch.uint8)),
            lambda: sp.sp24_gemm_fp8(*w, 17, codes[:, :48], scales), lambda: sp.sp24_gemm_fp8(w[0], w[1][:-1], w[2], 8, codes, scales),
            lambda: sp.sp24_gemm_fp8(*w, 300, codes, scales), lambda: sp.sp24_gemm_fp8(*w, 8, codes, scales[:2]),
            lambda: sp.sp24_gemm_fp8(*w, 8, codes, scales, out=torch.zeros(4, 9, device="cuda", dtype=torch.bfloat16)),
            lambda: sp.sp24_grad_weight_fp8(dy.float(), codes, scales), lambda: sp.sp24_grad_weight_fp8(dy[:3], codes, scales),
            lambda: sp.sp24_grad_weight_fp8(dy, codes, scales, meta=w[1][:-4]), lambda: sp.sp24_decompress_fp8(*w, 8, 144)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sp.sp24_quant_fp8(x[:, :40]), lambda: sp.sp24_quant_fp8(x.float()[:, 2:50]),
                 lambda: sp.sp24_rmsnorm_fp8(x, g, eps=-1.0), lambda: sp.sp24_gemm_fp8(*w, 8, codes, scales, out_dtype=torch.float32),
                 lambda: sp.sp24_decompress_fp8(*w, 8, 64, out_dtype=torch.float16),
                 lambda: sp.sp24_grad_weight_fp8(dy[:, :4], codes, scales, out_dtype=torch.float16)):
        with pytest.raises(sp.Sp24Error):
            call()
