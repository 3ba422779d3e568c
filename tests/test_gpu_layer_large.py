"""Layer operators where sizes change how they work: outputs past the caches, pitches and offsets beyond 32 bits, batches beyond one
launch, the gradient's ways of splitting its tokens, and calls at once on two streams."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import layer_ref as ref
from tests import test_gpu_layer_adamw as adam
from tests import test_gpu_layer_back as back
from tests.gpu_util import require_gpu, say
from tests.test_gpu_layer_products import BF16, FP16, FP32, check, fused, rand, weight, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("out", [FP32, BF16])
@pytest.mark.parametrize("layout,M,N", [("token", 8192, 4100), ("token", 8200, 4224), ("feature", 4100, 8192), ("feature", 8320, 4104)])
def test_bf16_output_past_the_caches(layout, M, N, out):
    """64 MB and more of Y, whole blocks and cut ones: elsewhere, and in the residual's place."""
    say(f"bf16 fused large {layout} {M} N={N} {out}")
    K = 64
    values, meta = weight(1, M, K)
    X = rand(2, *((N, K) if layout == "token" else (K, N)), dtype=BF16)
    bias = rand(3, M)
    z32 = sp.sp24_gemm_bf16_ex(values, meta, M, X, layout=layout) + (bias if layout == "token" else bias[:, None])
    R = rand(4, *z32.shape, dtype=out)
    Y, Z = fused(values, meta, M, X, layout, out, bias=bias, activation="gelu", residual=R, preact=True)
    assert torch.equal(Z, z32.to(out))
    check(Y, z32, "gelu", R)
    fused(values, meta, M, X, layout, out, bias=bias, activation="gelu", residual=R, out=R)
    assert torch.equal(R, Y)


@pytest.mark.parametrize("M,N", [(8192, 4100), (8200, 4224)])
@pytest.mark.parametrize("out", [BF16, FP16])
def test_fp8_output_past_the_caches(M, N, out):
    say(f"fp8 fused large {M} N={N} {out}")
    K = 144
    W, X = sp.sp24_prune_mask(whole(1, M, K), 2)[1], whole(2, N, K)
    w, (codes, scales) = sp.sp24_prune_compress_fp8(W), sp.sp24_quant_fp8(X)
    bias, R = rand(3, M), rand(4, N, M, dtype=out)
    z32 = X @ W.t() + bias
    Y, Z = sp.sp24_gemm_fp8_fused(*w, M, codes, scales, bias=bias, activation="silu", residual=R, preact=True, out_dtype=out)
    assert torch.equal(Z, z32.to(out))
    check(Y, z32, "silu", R)
    sp.sp24_gemm_fp8_fused(*w, M, codes, scales, bias=bias, activation="silu", residual=R, out=R)
    assert torch.equal(R, Y)


def test_fp8_far_apart_scales_among_many_tiles():
    """16576 tiles, more than 64 a workgroup, some of them summed again from memory; the residual's place is the output's."""
    say("fp8 fused, far apart scales, 16576 tiles")
    M, K, N = 28672, 144, 37888
    W, X = sp.sp24_prune_mask(whole(1, M, K), 2)[1], whole(2, N, K)
    far = [5, 20_000, 37_000, 37_800]
    X[far, :128] *= 2.0 ** 70
    X[far, 128:] *= 2.0 ** -30
    w, (codes, scales) = sp.sp24_prune_compress_fp8(W), sp.sp24_quant_fp8(X)
    R = torch.empty(N, M, dtype=BF16, device="cuda")
    for i, part in enumerate(R.split(4096)):
        part.copy_(rand(10 + i, *part.shape))
    Y = sp.sp24_gemm_fp8_fused(*w, M, codes, scales, activation="relu", residual=R)
    for i in (0, 18944, 36864):
        near = torch.tensor([n not in far for n in range(i, i + 512)], device="cuda")
        check(Y[i:i + 512][near], X[i:i + 512][near] @ W.t(), "relu", R[i:i + 512][near])
    sp.sp24_gemm_fp8_fused(*w, M, codes, scales, activation="relu", residual=R, out=R)
    assert torch.equal(R, Y)


@pytest.mark.parametrize("which", ["Y", "Z", "R"])
@pytest.mark.parametrize("layout,M,N", [("token", 260, 17), ("token", 256, 72), ("feature", 72, 136), ("feature", 40, 24)])
def test_rows_of_128_megabytes(layout, M, N, which):
    """One of Y, Z and R with rows so far apart that 16 of them pass 2^31 bytes."""
    say(f"bf16 fused pitch 2^25 {layout} {M} N={N} {which}")
    K, pitch = 128, 1 << 25
    values, meta = weight(1, M, K)
    X = rand(2, *((N, K) if layout == "token" else (K, N)), dtype=BF16)
    bias = rand(3, M)
    plain = sp.sp24_gemm_bf16_ex(values, meta, M, X, layout=layout)
    rows, cols = plain.shape
    wide = torch.empty((rows - 1) * pitch + cols, device="cuda").as_strided((rows, cols), (pitch, 1))
    ops = {k: torch.empty_like(plain) for k in "YZR"}
    ops[which] = wide
    ops["R"].copy_(rand(4, rows, cols))
    fused(values, meta, M, X, layout, FP32, bias=bias, activation="silu", residual=ops["R"], preact=ops["Z"], out=ops["Y"])
    z32 = plain + (bias if layout == "token" else bias[:, None])
    assert torch.equal(ops["Z"], z32)
    check(ops["Y"], z32, "silu", ops["R"])


@pytest.mark.parametrize("layout,M,N", [("token", 512, 4_300_005), ("feature", 33_000, 70_000)])
def test_bf16_offsets_past_32_bits(layout, M, N):
    """Y, Z and R of more than 4 GB each: their first and last rows."""
    say(f"bf16 fused {layout} {M} N={N}")
    K = 64
    values, meta = weight(1, M, K)
    X = rand(2, *((N, K) if layout == "token" else (K, N)), dtype=BF16)
    bias = rand(3, M)
    R = torch.empty((N, M) if layout == "token" else (M, N), dtype=BF16, device="cuda")
    for i, part in enumerate(R.split(4096 if layout == "feature" else 1 << 20)):
        part.copy_(rand(10 + i, *part.shape))
    Y, Z = fused(values, meta, M, X, layout, BF16, bias=bias, activation="gelu", residual=R, preact=True)
    whole_z = None if layout == "token" else sp.sp24_gemm_bf16_ex(values, meta, M, X, layout=layout)
    for s in (slice(0, 300), slice(-300, None)):
        if layout == "token":
            z32 = sp.sp24_gemm_bf16_ex(values, meta, M, X[s], layout=layout) + bias
        else:
            z32 = whole_z[s] + bias[s][:, None]
        assert torch.equal(Z[s], z32.to(BF16))
        check(Y[s], z32, "gelu", R[s])


@pytest.mark.parametrize("layout,N", [("token", 2), ("token", 24), ("token", 72), ("feature", 2), ("feature", 24), ("feature", 72)])
def test_batches_beyond_one_launch(layout, N):
    """65537 products: every entry has its own residual and pre-activation."""
    say(f"bf16 fused 65537 entries {layout} N={N}")
    M, K, B = 24, 16, 65537
    values, meta = weight(1, M, K)
    X = rand(2, B, *((N, K) if layout == "token" else (K, (N + 7) // 8 * 8)), dtype=BF16)[..., :K if layout == "token" else N]
    bias = rand(3, M)
    shape = (N, M) if layout == "token" else (M, N)
    R = rand(4, B, *shape)
    Y, Z = fused(values, meta, M, X, layout, FP32, bias=bias, activation="relu", residual=R, preact=True)
    z32 = sp.sp24_gemm_bf16_ex(values, meta, M, X, layout=layout) + (bias if layout == "token" else bias[:, None])
    assert torch.equal(Z, z32)
    check(Y, z32, "relu", R)


# ---------------------------------------------------------------- the epilogue's gradient

@pytest.mark.parametrize("M", [8191, 8192])
@pytest.mark.parametrize("N", [256, 257, 512, 513, 2500])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradient_where_its_split_changes(N, M, dtype):
    say(f"epilogue gradient {N}x{M} {dtype}")
    dY, Z = back.rand(N, N, M, dtype=dtype), back.rand(M, N, M, dtype=dtype, scale=2.0)
    dZ, dbias = sp.sp24_epilogue_backward(dY, Z, "gelu")
    back.check(dZ, dbias, dY, Z, "gelu")
    _, alone = sp.sp24_epilogue_backward(dY)
    assert ((alone.double() - dY.double().sum(0)).abs() <= N * ref.U * dY.double().abs().sum(0)).all()


@pytest.mark.parametrize("N,M", [(2_200_003, 1000), (520, 1 << 22)])
def test_gradient_offsets_past_32_bits(N, M):
    """dY, Z and dZ of more than 4 GB: the first and last rows, and the bias's gradient of the last columns."""
    say(f"epilogue gradient {N}x{M}")
    dY, Z = (torch.empty(N, M, dtype=BF16, device="cuda") for _ in range(2))
    for seed, t in enumerate((dY, Z)):
        for i, part in enumerate(t.split(max((1 << 28) // M, 1))):
            part.copy_(back.rand(2 * i + seed, *part.shape))
    dZ, dbias = sp.sp24_epilogue_backward(dY, Z, "silu")
    for s in (slice(0, 4), slice(-4, None)):
        back.check(dZ[s], None, dY[s], Z[s], "silu")
    cols = slice(M - 40, M)
    back.check(dZ[:, cols], dbias[cols], dY[:, cols], Z[:, cols], "silu")


def test_gradients_on_two_streams():
    """Two gradients at once, each with sums of its own."""
    say("epilogue gradients on two streams")
    ins = [(back.rand(i, 3000 + i, 1000, dtype=BF16), back.rand(10 + i, 3000 + i, 1000, dtype=BF16)) for i in range(2)]
    want = [sp.sp24_epilogue_backward(*x, "gelu") for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sp.sp24_epilogue_backward(*ins[i], "gelu"))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for pair in g for a, b in zip(pair, w))


# ---------------------------------------------------------------- AdamW

@pytest.mark.parametrize("bits,start", [(32, 1 << 30), (8, 1 << 32)])
def test_adamw_offsets_past_32_bits(bits, start):
    """Weights and moments beyond 4 GB: the last 1035 elements of a tensor of zeros; with 8 bits their random bits are those of their
    positions, of which the higher 32 bits enter the key."""
    say(f"adamw {start} elements and more, {bits} bits")
    n, first = start + 5003, start + 31 * 128
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    p[first:], g[first:] = adam.rand(1, n - first), adam.rand(2, n - first, scale=1e-2)
    state = sp.sp24_adamw_state(p, bits)
    want, off, new = adam.expect(p[first:], g[first:], sp.sp24_adamw_state(p[first:], bits), step=1, seed=3)
    if bits == 8:
        zeros = np.zeros(n - first, np.float32)
        m, v = ref.moments(zeros, zeros, adam.host(g[first:]), 0.9, 0.999)
        with np.errstate(over="ignore"):
            key = ref.mix(ref.mix(ref.mix(ref.mix(np.uint32(3)) ^ np.uint32(0)) ^ np.uint32(1)))
            assert ref.random_words(3, 1, 0, 1)[0] == ref.mix(key)
            r = ref.mix(np.arange(first, n).astype(np.uint32) * np.uint32(0xBB67AE85) + (key + np.uint32(start >> 32) * np.uint32(0x9E3779B9)))
        new = (*ref.first_codes(m, r & 0xFFFF), *ref.second_codes(v, r >> 16))
    sp.sp24_adamw([p], [g], [state], 1, seed=3, **adam.HYPER)
    end = [t[first:] if t.numel() == n else t[first // 128:] for t in state]
    adam.check(p[first:], end, want, off, new)
    assert not p[:first].any()


def test_adamw_states_must_be_lists():
    say("adamw states of a wrong kind")
    p = torch.zeros(64, device="cuda")
    for bad in (p, None, 3, (p,), (p, p, p), [[p, p], p]):
        with pytest.raises((TypeError, ValueError)):
            sp.sp24_adamw([p], [torch.zeros_like(p)], [bad], 1)
