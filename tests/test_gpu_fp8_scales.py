"""Scales of the 8-bit product at their extremes. Codes are small whole numbers, so every block's sum is exact in the
matrix instruction and in fp32."""
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
