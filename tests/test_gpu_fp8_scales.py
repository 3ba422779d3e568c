"""Scales of the 8-bit product at their extremes: NaN, far apart in either order, 2^-127, and those of blocks of zeros.

Codes are small whole numbers, so every block's sum is exact in the matrix instruction and in fp32. Where all that a
row of the weight keeps lies in blocks of one unit, its outputs are the rounded 64-bit result bit for bit, whatever
the other blocks' scales are: what they add is zero. Elsewhere the largest unit decides and the result is within the
roundings of T fp32 additions and of the output."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import fp8_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

# (M, N): few tokens with one fragment, with three, with four; many tokens in tiles 128 wide, 256 wide, and several
# 128-wide tiles a workgroup (on 256 compute units)
SIZES = [(260, 3), (300, 40), (515, 150), (4100, 1000), (8200, 1030), (4100, 4090)]
K = 1168  # nine blocks and one of 16 columns
T = 10


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def case(M, N, seed=0):
    """(w, x): 2:4 weights in -3..3 and inputs in -4..4, as fp64 arrays without their scales."""
    rng = np.random.default_rng(M + 3 * N + seed)
    w = rng.integers(-3, 4, (M, K)).astype(np.float64)
    return w * ref.keep2(w), rng.integers(-4, 5, (N, K)).astype(np.float64)


def e8m0(byte):
    return torch.from_numpy(np.ascontiguousarray(byte, dtype=np.uint8)).cuda().view(torch.float8_e8m0fnu)


def weight(w, sw):
    """The compressed weight with codes w and scale bytes sw."""
    v, m, s = sp.sp24_prune_compress_fp8(torch.from_numpy(w).float().cuda())
    # the compressor's codes use up to 448 units: back to codes of w itself (blocks of zeros stay zeros)
    tiles = -(-w.shape[0] // 16)
    unit = s.float().repeat_interleave(8, 0)[:tiles].unsqueeze(2).expand(-1, -1, 1024).reshape(-1)
    return (v.float() * unit).to(torch.float8_e4m3fn), m, e8m0(sw)


def product(w, sw, x, sx, dtype=torch.bfloat16):
    codes = torch.from_numpy(x).to(torch.float8_e4m3fn).cuda()
    return ref.f64(sp.sp24_gemm_fp8(*weight(w, sw), w.shape[0], codes, e8m0(sx), out_dtype=dtype))


def block_of_columns(b):
    return slice(128 * b, min(K, 128 * b + 128))


def scaled(w, sw, x, sx):
    """The operands with their scales, in 64 bits."""
    rows = np.repeat(2.0 ** (sw.astype(np.float64) - 127), 128, 0)[:w.shape[0]]
    return w * np.repeat(rows, 128, 1)[:, :K], x * np.repeat(2.0 ** (sx.astype(np.float64) - 127), 128, 1)[:, :K]


def rounded(y, dtype=torch.bfloat16):
    return ref.f64(torch.from_numpy(y).to(dtype))


def scale_bytes(M, N):
    return np.full((-(-M // 128), T), 127), np.full((N, T), 127)


@pytest.mark.parametrize("M,N", SIZES)
def test_nan_weight_scale(M, N):
    """A NaN scale of the weight makes its 128 output channels NaN, as it makes them in the decompressed weight."""
    say(f"gemm fp8 NaN weight scale {M} N {N}")
    w, x = case(M, N)
    sw, sx = scale_bytes(M, N)
    sw[1, 4] = 255
    bad = np.zeros(M, bool)
    bad[128:256] = True
    got = product(w, sw, x, sx)
    assert np.isnan(got[:, bad]).all()
    assert np.array_equal(got[:, ~bad], rounded(x @ w.T)[:, ~bad])
    dense = ref.f64(sp.sp24_decompress_fp8(*weight(w, sw), M, K, torch.float32))
    assert np.isnan(dense[128:256, 512:640]).any() and not np.isnan(dense[~bad]).any()
    assert not np.isnan(np.delete(dense, np.s_[512:640], 1)).any()


# exponents of the scales of x in blocks 0 .. 9
FAR = {
    "large first": [80] + [0] * 9,
    "large last": [-70] * 9 + [70],
    "large in the middle": [0] * 5 + [90] + [0] * 4,
    "small last": [0] * 9 + [-80],
    "rising": [-90 + 20 * b for b in range(10)],
    "falling": [90 - 20 * b for b in range(10)],
    "up and down": [0, 70, -70, 70, -70, 0, 100, -100, 0, 65],
    "across the limit": [0, 64, 0, 65, 0, -64, 0, -65, 63, 0],
}


@pytest.mark.parametrize("exponents", FAR.values(), ids=FAR.keys())
@pytest.mark.parametrize("M,N", SIZES)
def test_scales_far_apart(M, N, exponents):
    """Some tokens with such scales among ordinary ones. Row m of the weight keeps only block m % 11 (or, at 10, all)."""
    say(f"gemm fp8 far scales {M} N {N} {exponents}")
    w, x = case(M, N, 1)
    which = np.arange(M) % 11
    for b in range(T):
        w[:, block_of_columns(b)] *= ((which == b) | (which == 10))[:, None]
    sw, sx = scale_bytes(M, N)
    far = np.arange(N) % 97 == 2
    sx[far] += np.array(exponents)
    got = product(w, sw, x, sx)
    wf, xf = scaled(w, sw, x, sx)
    want = xf @ wf.T
    assert np.array_equal(got[:, which < 10], rounded(want)[:, which < 10])
    assert np.array_equal(got[~far], rounded(want)[~far])
    bound = 1.01 * ref.UB * np.abs(want) + (T + 8) * ref.U32 * (np.abs(xf) @ np.abs(wf).T)
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("M,N", SIZES)
def test_blocks_of_zeros(M, N):
    """Zero blocks of a token or a weight carry the least scale, 2^-127, wherever they lie; a token of zeros."""
    say(f"gemm fp8 zero blocks {M} N {N}")
    w, x = case(M, N, 2)
    sw, sx = scale_bytes(M, N)
    for n, blocks in ((0, [0]), (1, [0, 1, 2]), (2, [9]), (N - 1, [4, 8]), (N // 2, range(T))):
        for b in blocks:
            x[n, block_of_columns(b)] = 0
            sx[n, b] = 0
    for m, b in ((0, 0), (0, 5), (1, 9), (sw.shape[0] - 1, 3)):
        w[128 * m:128 * m + 128, block_of_columns(b)] = 0
        sw[m, b] = 0
    assert np.array_equal(product(w, sw, x, sx), rounded(x @ w.T))


@pytest.mark.parametrize("M,N", SIZES)
def test_least_scales(M, N):
    """2^-127 on blocks that hold something, beside ordinary ones."""
    say(f"gemm fp8 least scales {M} N {N}")
    w, x = case(M, N, 3)
    which = np.arange(M) % 2
    for b in range(T):
        w[:, block_of_columns(b)] *= (which == b % 2)[:, None]
    sw, sx = scale_bytes(M, N)
    sx[1::3, 1::2] = 0  # of rows with which == 1: their results are whole numbers times 2^-127
    sw[:, 1::2] = 137   # 2^10
    got = product(w, sw, x, sx)
    wf, xf = scaled(w, sw, x, sx)
    assert np.array_equal(got, rounded(xf @ wf.T))


def test_far_apart_among_many_tiles():
    """More than 64 tiles a wave, of which some are summed again."""
    M, N, k = 4096, 280000, 272
    say(f"gemm fp8 far scales among many tiles {M}x{k} N {N}")
    rng = np.random.default_rng(5)
    w = rng.integers(-3, 4, (M, k)).astype(np.float64)
    w *= ref.keep2(w)
    w[::2, 128:256] = 0
    x = rng.integers(-4, 5, (N, k)).astype(np.float32)
    sx = np.full((N, 3), 127)
    far = np.arange(N) % 20011 == 7
    sx[far, 1] = 227
    sw = np.full((M // 128, 3), 127)
    v, m, s = sp.sp24_prune_compress_fp8(torch.from_numpy(w).float().cuda())
    unit = s.float().repeat_interleave(8, 0).unsqueeze(2).expand(-1, -1, 1024).reshape(-1)
    codes = torch.from_numpy(x).cuda().to(torch.float8_e4m3fn)
    y = sp.sp24_gemm_fp8((v.float() * unit).to(torch.float8_e4m3fn), m, e8m0(sw), M, codes, e8m0(sx))
    at = np.unique(np.concatenate([np.flatnonzero(far), np.flatnonzero(far) + 1, rng.integers(0, N, 500)]))
    got = ref.f64(y[torch.from_numpy(at).cuda()])
    big = np.repeat(2.0 ** (sx[at].astype(np.float64) - 127), 128, 1)[:, :k] * x[at]
    want = big @ w.T
    assert np.array_equal(got[:, ::2], rounded(want)[:, ::2])
    assert (np.abs(got - want) <= 1.01 * ref.UB * np.abs(want) + 20 * ref.U32 * (np.abs(big) @ np.abs(w).T)).all()
