"""The bias's gradient where a wrong part, a row missed or counted twice, would show: whole numbers, whose fp32 sums are exact in any
order (every partial sum is below 2^24), and random ones within the depth of the sums that are really made.

The depth, from the kernel's split: eight threads lie along a row (64 from 8192 columns and 513 rows on), so 32 (4) rows go through a
workgroup at a time; a thread adds its rows of the part, the workgroup its 32 (4) sums, and where there are parts 16 threads
a column take every 16th and add their 16 sums."""
import ctypes

import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import layer_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
# one part; few; 79, 129 and 128 parts, the last one cut; long rows split; the last column block cut
SIZES = [(1, 1), (31, 9), (197, 768), (257, 1000), (512, 8200), (5000, 16), (8200, 40), (6304, 768), (513, 8199), (1030, 28672), (16391, 8192), (70001, 130)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def parts_of(N, M):
    n = ctypes.c_int64()
    assert sp.load_library().sp24_epilogue_backward_bytes(N, M, ctypes.byref(n)) == 0
    return max(1, n.value // (4 * M))


def whole(seed, N, M, dtype, most=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, (N, M), generator=g, device="cuda", dtype=torch.int8).to(dtype)


def column_sums(x):
    s = torch.zeros(x.shape[1], dtype=torch.float64, device="cuda")
    for rows in x.split(50000):
        s += rows.double().sum(0)
    return s


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("N,M", SIZES)
def test_whole_numbers(N, M, dtype):
    """z of 200 and -200: slopes of exactly one and zero with every activation."""
    say(f"bias gradient of whole numbers {N}x{M} {dtype}, {parts_of(N, M)} parts")
    dY = whole(N, N, M, dtype)
    _, dbias = sp.sp24_epilogue_backward(dY)
    assert torch.equal(dbias.double(), column_sums(dY))
    on = whole(M, N, M, dtype, 1) > 0
    Z = torch.where(on, 200.0, -200.0).to(dtype)
    want = torch.where(on, dY, 0)
    for act in ("gelu", "relu", "silu"):
        dZ, dbias = sp.sp24_epilogue_backward(dY, Z, act)
        assert torch.equal(dZ, want) and torch.equal(dbias.double(), column_sums(want))


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("N,M", [(2_200_003, 1000), (262_147, 8200)])
def test_whole_numbers_past_4_gb(N, M, act):
    """2.2 million times 4 is below 2^24."""
    say(f"bias gradient of whole numbers {N}x{M} {act}, {parts_of(N, M)} parts")
    assert N * M * 2 > 1 << 32 and parts_of(N, M) > 16 and 4 * N < 1 << 24
    dY = whole(3, N, M, BF16)
    if act == "none":
        _, dbias = sp.sp24_epilogue_backward(dY)
        assert torch.equal(dbias.double(), column_sums(dY))
        return
    Z = whole(4, N, M, BF16, 1)
    on = Z > 0
    Z.fill_(-200.0).masked_fill_(on, 200.0)
    dZ, dbias = sp.sp24_epilogue_backward(dY, Z, act)
    dY.masked_fill_(~on, 0)
    assert torch.equal(dZ, dY) and torch.equal(dbias.double(), column_sums(dY))


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("N,M", [(5000, 16), (8200, 40), (6304, 768), (1030, 28672), (70001, 130), (2_200_003, 100)])
def test_depth_of_the_sums(N, M, act):
    """Each of d additions in a chain is off by U of a partial sum at most sum |dZ|: d U sum |dZ|, besides the products' own errors."""
    parts = parts_of(N, M)
    down = 4 if M >= 8192 and N > 512 else 32
    rows = -(-(-(-N // parts)) // down) * down  # a part's, a whole number of rounds
    depth = -(-rows // down) + down + (-(-parts // 16) + 15 if parts > 1 else 0)
    say(f"bias gradient {N}x{M} {act}: {parts} parts, depth {depth}")
    g = torch.Generator(device="cuda").manual_seed(N)
    dY, Z = torch.randn(N, M, generator=g, device="cuda"), 2 * torch.randn(N, M, generator=g, device="cuda")
    _, dbias = sp.sp24_epilogue_backward(dY) if act == "none" else sp.sp24_epilogue_backward(dY, Z, act)
    want, size, off = (torch.zeros(M, dtype=torch.float64, device="cuda") for _ in range(3))
    for dy, z in zip(dY.split(50000), Z.split(50000)):
        dy, z = dy.double(), z.double()
        if act == "none":
            want += dy.sum(0)
            size += dy.abs().sum(0)
            continue
        dz = dy * ref.slope(z, act)
        want += dz.sum(0)
        size += dz.abs().sum(0)
        off += (dy.abs() * ref.slope_error(z, act) + ref.U * dz.abs()).sum(0)
    bound = off + depth * ref.U * (size + off)
    assert ((dbias.double() - want).abs() <= bound).all()
    if act == "none" and N < 100_000:
        assert (bound < 0.5 * dY.abs().mean(0)).all()  # below half an average row: one that is missed shows
