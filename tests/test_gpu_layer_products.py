"""The products with a fused epilogue. What they sum is what the plain products sum, to the bit, so z = acc + bias is compared
exactly (bf16: from the plain product's fp32 result; 8 bits: from whole numbers, whose sums are exact), and Y with the
activation of that z in 64 bits: within the activation's error, one fp32 rounding for the residual's sum, and one to Y's type."""
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import layer_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rand(seed, *shape, dtype=FP32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def weight(seed, M, K):
    return sp.sp24_prune_compress(rand(seed, M, K, dtype=BF16, scale=(2.0 / K) ** 0.5))


def padded(shape, extra, dtype, fill=float("nan")):
    """(the whole buffer, a view of `shape` in it whose rows are `extra` elements longer)."""
    buf = torch.full((*shape[:-1], shape[-1] + extra), fill, dtype=dtype, device="cuda")
    return buf, buf[..., :shape[-1]]


def check(Y, z, act, residual):
    """Y against act(z) + residual, z fp32 exactly."""
    z = z.double()
    a = ref.act(z, act)
    want = a if residual is None else a + residual.double()
    # |y32 - want| <= act's error + U |y32|; Y is y32 rounded
    off32 = ref.act_error(z, act) + (0 if residual is None else ref.U * want.abs())
    bound = off32 + (want.abs() + off32) * (0 if Y.dtype is FP32 else ref.UNIT[Y.dtype]) * 1.0001 + 1e-37
    if Y.dtype is FP16:
        bound = bound + 2.0 ** -25  # below the least normal number
    fine = torch.isfinite(want)
    got = Y.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert (((got - want).abs() <= bound) | ~fine | (want.abs() > torch.finfo(Y.dtype).max)).all()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])


def fused(values, meta, M, X, layout, out_dtype, **kw):
    return sp.sp24_gemm_bf16_fused(values, meta, M, X, layout=layout, out_dtype=out_dtype, **kw)


# token-major: (M, K, N, extra elements in X's rows); between them every kernel: through LDS up to 16 tokens, from registers up
# to 64 and with rows of X at any element, the tiles of both widths with one and several a workgroup, and the general one
TOKEN = [(1, 16, 1, 0), (48, 64, 1, 0), (300, 80, 2, 0), (3000, 128, 1, 8), (640, 144, 7, 0), (4112, 64, 5, 0), (257, 192, 16, 0),
         (4200, 64, 16, 0), (100, 64, 20, 0), (9000, 64, 33, 0), (33, 64, 64, 0), (65, 48, 3, 1), (1000, 64, 40, 3),
         (256, 64, 65, 0), (255, 128, 200, 8), (1, 64, 70, 0), (130, 192, 129, 0), (77, 80, 100, 0), (50, 64, 130, 1),
         (4100, 2048, 1030, 0), (2050, 128, 8330, 0), (8190, 256, 4090, 0), (512, 64, 256, 0)]
FEATURE = [(1, 16, 1, 0), (300, 64, 1, 0), (2000, 128, 1, 7), (100, 64, 8, 0), (65, 80, 24, 0), (33, 64, 33, 0), (9000, 64, 64, 0),
           (700, 128, 40, 8), (256, 64, 72, 0), (255, 80, 200, 0), (130, 64, 136, 8), (64, 64, 75, 0), (1, 16, 80, 0),
           (4100, 2048, 1032, 0), (2050, 128, 8328, 0), (8190, 256, 4096, 0)]
CASES = [("token", *c) for c in TOKEN] + [("feature", *c) for c in FEATURE]


@pytest.mark.parametrize("layout,M,K,N,extra", CASES)
def test_bf16_every_kernel(layout, M, K, N, extra):
    say(f"bf16 fused {layout} {M}x{K} N={N} extra {extra}")
    values, meta = weight(M + K, M, K)
    _, X = padded((N, K) if layout == "token" else (K, N), extra, BF16, 0.0)
    X.copy_(rand(N, *X.shape))
    bias = rand(1, M)
    plain = sp.sp24_gemm_bf16_ex(values, meta, M, X, layout=layout)
    z32 = plain + (bias if layout == "token" else bias[:, None])
    for out in (FP32, BF16):
        R = rand(2, *plain.shape, dtype=out)
        for act in ref.ACTIVATIONS:
            Y, Z = fused(values, meta, M, X, layout, out, bias=bias, activation=act, residual=R, preact=True)
            assert torch.equal(Z, z32.to(out)), act
            check(Y, z32, act, R)
    # parts left out
    assert torch.equal(fused(values, meta, M, X, layout, FP32), plain)
    Y = fused(values, meta, M, X, layout, BF16, activation="gelu")
    check(Y, plain, "gelu", None)
    Y = fused(values, meta, M, X, layout, FP32, residual=plain)
    assert torch.equal(Y, plain + plain)


@pytest.mark.parametrize("out", [FP32, BF16])
@pytest.mark.parametrize("layout,M,K,N", [("token", 260, 128, 140), ("token", 130, 128, 9), ("token", 70, 64, 30), ("token", 90, 80, 80),
                                          ("feature", 260, 128, 136), ("feature", 130, 64, 24), ("feature", 90, 80, 75)])
@pytest.mark.parametrize("pads", [(0, 0, 0), (1, 2, 3), (8, 8, 8), (5, 0, 16)])
def test_bf16_pitches_and_surroundings(layout, M, K, N, out, pads):
    """Pitches of their own for Y, Z and R; what lies between the rows stays as it was."""
    say(f"bf16 fused pitches {layout} {M}x{K} N={N} {out} {pads}")
    values, meta = weight(5, M, K)
    X = rand(6, *((N, K) if layout == "token" else (K, N)), dtype=BF16)
    bias = rand(7, M)
    shape = (N, M) if layout == "token" else (M, N)
    (by, Y), (bz, Z), (br, R) = (padded(shape, p, out) for p in pads)
    R.copy_(rand(8, *shape))
    got = fused(values, meta, M, X, layout, out, bias=bias, activation="silu", residual=R, preact=Z, out=Y)
    assert got[0] is Y or got[0].data_ptr() == Y.data_ptr()
    plain = sp.sp24_gemm_bf16_ex(values, meta, M, X, layout=layout)
    z32 = plain + (bias if layout == "token" else bias[:, None])
    assert torch.equal(Z, z32.to(out))
    check(Y, z32, "silu", R)
    for buf, p in zip((by, bz, br), pads):
        assert p == 0 or torch.isnan(buf[..., shape[-1]:]).all()


@pytest.mark.parametrize("layout,M,K,N", [("token", 260, 128, 140), ("token", 130, 128, 9), ("token", 70, 64, 30), ("feature", 260, 128, 136),
                                          ("feature", 64, 64, 24), ("feature", 90, 80, 76)])
@pytest.mark.parametrize("out", [FP32, BF16])
def test_bf16_batches(layout, M, K, N, out):
    """Entries one by one are the batch; a residual shared by all through a stride of 0; the residual updated in place."""
    say(f"bf16 fused batch {layout} {M}x{K} N={N} {out}")
    values, meta = weight(9, M, K)
    X = rand(10, 3, *((N, K) if layout == "token" else (K, N)), dtype=BF16)
    bias, shape = rand(11, M), ((N, M) if layout == "token" else (M, N))
    if shape[0] * shape[1] * (2 if out is BF16 else 4) % 16:
        with pytest.raises(sp.Sp24Error):
            fused(values, meta, M, X, layout, out)
        return
    R = rand(12, 3, *shape, dtype=out)
    shared = R[:1].expand(3, *shape)
    Y, Z = fused(values, meta, M, X, layout, out, bias=bias, activation="gelu", residual=R, preact=True)
    S = fused(values, meta, M, X, layout, out, bias=bias, activation="gelu", residual=shared)
    inplace = R.clone()
    assert fused(values, meta, M, X, layout, out, bias=bias, activation="gelu", residual=inplace, out=inplace).data_ptr() == inplace.data_ptr()
    assert torch.equal(inplace, Y)
    for b in range(3):
        y, z = fused(values, meta, M, X[b], layout, out, bias=bias, activation="gelu", residual=R[b], preact=True)
        assert torch.equal(Y[b], y) and torch.equal(Z[b], z)
        assert torch.equal(S[b], fused(values, meta, M, X[b], layout, out, bias=bias, activation="gelu", residual=R[0]))


def special_values():
    v = torch.cat([torch.linspace(-30, 30, 3001), torch.logspace(-38, 38, 200), -torch.logspace(-38, 38, 200), torch.linspace(-90, -85, 101),
                   torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 3.4e38, -3.4e38, 1e-45, -1e-45])])
    return v.cuda()


@pytest.mark.parametrize("act", ref.ACTIVATIONS)
@pytest.mark.parametrize("layout,N", [("token", 1), ("token", 24), ("token", 80), ("feature", 72), ("feature", 8)])
def test_activations_over_their_range(act, layout, N):
    """Weights of zeros: z is the bias, infinities and NaN among it."""
    say(f"activation {act} {layout} N={N}")
    bias = special_values()
    M = bias.numel()
    values, meta = sp.sp24_prune_compress(torch.zeros(M, 64, dtype=BF16, device="cuda"))
    X = torch.ones((N, 64) if layout == "token" else (64, N), dtype=BF16, device="cuda")
    for out in (FP32, BF16):
        Y, Z = fused(values, meta, M, X, layout, out, bias=bias, activation=act, preact=True)
        z = (bias if layout == "token" else bias[:, None]).expand_as(Y)
        assert torch.equal(torch.nan_to_num(Z), torch.nan_to_num(z.to(out)))
        check(Y, z, act, None)


def test_infinite_and_nan_residuals():
    say("residual infinities")
    M, K, N = 256, 64, 128
    values, meta = weight(1, M, K)
    X = rand(2, N, K, dtype=BF16)
    R = rand(3, N, M)
    R[0, 0], R[1, 1], R[2, 2] = float("inf"), -float("inf"), float("nan")
    Y = fused(values, meta, M, X, "token", FP32, activation="relu", residual=R)
    check(Y, sp.sp24_gemm_bf16_ex(values, meta, M, X, layout="token"), "relu", R)
    assert torch.isinf(Y).sum() == 2 and torch.isnan(Y).sum() == 1


# ---------------------------------------------------------------- 8 bits

def whole(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda").float()


FP8_SIZES = [(1, 16, 1), (100, 144, 1), (4112, 128, 3), (300, 272, 8), (4100, 256, 16), (9000, 128, 9), (500, 400, 30), (3000, 128, 48), (129, 128, 64),
             (256, 128, 190), (30000, 128, 100), (1030, 528, 1500), (2049, 128, 9000), (4096, 1024, 5000), (8190, 256, 4090)]


@pytest.mark.parametrize("M,K,N", FP8_SIZES)
def test_fp8_every_kernel(M, K, N):
    """Whole numbers up to 3: their products and sums below 2^24 are exact in any order."""
    say(f"fp8 fused {M}x{K} N={N}")
    W, X = sp.sp24_prune_mask(whole(M, M, K), 2)[1], whole(N, N, K)
    w, (codes, scales) = sp.sp24_prune_compress_fp8(W), sp.sp24_quant_fp8(X)
    assert torch.equal(sp.sp24_decompress_fp8(*w, M, K, FP32), W)
    acc = X @ W.t()
    bias = rand(4, M)
    z32 = acc + bias
    for out in (BF16, FP16):
        R = rand(5, N, M, dtype=out)
        for act in ref.ACTIVATIONS:
            Y, Z = sp.sp24_gemm_fp8_fused(*w, M, codes, scales, bias=bias, activation=act, residual=R, preact=True, out_dtype=out)
            assert torch.equal(Z, z32.to(out)), act
            check(Y, z32, act, R)
        assert torch.equal(sp.sp24_gemm_fp8_fused(*w, M, codes, scales, out_dtype=out), sp.sp24_gemm_fp8(*w, M, codes, scales, out_dtype=out))
        check(sp.sp24_gemm_fp8_fused(*w, M, codes, scales, activation="silu", out_dtype=out), acc, "silu", None)


@pytest.mark.parametrize("M,K,N", [(260, 144, 200), (9000, 128, 300), (130, 128, 9), (70, 272, 40)])
@pytest.mark.parametrize("pads", [(1, 2, 3), (8, 8, 8), (5, 0, 16)])
def test_fp8_pitches_and_in_place(M, K, N, pads):
    say(f"fp8 fused pitches {M}x{K} N={N} {pads}")
    W, X = sp.sp24_prune_mask(whole(M, M, K), 2)[1], whole(N, N, K)
    w, (codes, scales) = sp.sp24_prune_compress_fp8(W), sp.sp24_quant_fp8(X)
    bias = rand(4, M)
    (by, Y), (bz, Z), (br, R) = (padded((N, M), p, BF16) for p in pads)
    R.copy_(rand(8, N, M))
    sp.sp24_gemm_fp8_fused(*w, M, codes, scales, bias=bias, activation="gelu", residual=R, preact=Z, out=Y)
    z32 = X @ W.t() + bias
    assert torch.equal(Z, z32.to(BF16))
    check(Y, z32, "gelu", R)
    for buf, p in zip((by, bz, br), pads):
        assert p == 0 or torch.isnan(buf[:, M:]).all()
    sp.sp24_gemm_fp8_fused(*w, M, codes, scales, bias=bias, activation="gelu", residual=R, out=R)
    assert torch.equal(R, Y)
    assert br is None or pads[2] == 0 or torch.isnan(br[:, M:]).all()


@pytest.mark.parametrize("act", ref.ACTIVATIONS)
def test_fp8_scales_far_apart_and_nan(act):
    """Tokens whose blocks lie more than 2^64 apart (their tiles are summed again from memory), and NaN scales."""
    say(f"fp8 fused far apart {act}")
    M, K, N = 520, 384, 9000
    W = sp.sp24_prune_mask(whole(1, M, K), 2)[1]
    X = whole(2, N, K)
    X[5, :128] *= 2.0 ** 70
    X[5, 128:256] *= 2.0 ** -30
    X[8000, 256:] *= 2.0 ** -100
    X[17, 3] = float("nan")
    w, (codes, scales) = sp.sp24_prune_compress_fp8(W), sp.sp24_quant_fp8(X)
    bias, R = rand(3, M), rand(4, N, M, dtype=BF16)
    Y, Z = sp.sp24_gemm_fp8_fused(*w, M, codes, scales, bias=bias, activation=act, residual=R, preact=True)
    plain = sp.sp24_gemm_fp8(*w, M, codes, scales)
    assert torch.isnan(Y[17]).all() and torch.isnan(Z[17]).all()
    rows = torch.ones(N, dtype=torch.bool, device="cuda")
    rows[17] = False
    assert not torch.isnan(Y[rows]).any()
    assert torch.equal(sp.sp24_gemm_fp8_fused(*w, M, codes, scales, preact=True)[1][rows], plain[rows])
    rows[5] = rows[8000] = False
    z32 = X[rows] @ W.t() + bias
    assert torch.equal(Z[rows], z32.to(BF16))
    check(Y[rows], z32, act, R[rows])
    # the two rows: sums in 64 bits, each term's fp32 rounding at most 2^-24 of the largest
    for n in (5, 8000):
        z = X[n].double() @ W.t().double() + bias.double()
        near = z.abs() * (ref.UNIT[BF16] + 8 * ref.U) + 8 * ref.U * (X[n].double().abs() @ W.t().double().abs())
        assert ((Z[n].double() - z).abs() <= near).all()


# ---------------------------------------------------------------- graphs, streams, refusals

def test_products_captured_and_replayed():
    say("fused products in a graph")
    M, K = 1030, 256
    values, meta = weight(1, M, K)
    w8 = sp.sp24_prune_compress_fp8(rand(2, M, K, dtype=BF16))
    bias = rand(3, M)
    sizes = (1, 40, 300)
    xs = [rand(4, n, K, dtype=BF16) for n in sizes]
    q8 = [sp.sp24_quant_fp8(x) for x in xs]
    rs = [rand(5, n, M, dtype=BF16) for n in sizes]

    def run():
        got = []
        for x, (c, s), r in zip(xs, q8, rs):
            got += sp.sp24_gemm_bf16_fused(values, meta, M, x, bias, "gelu", r, True, "token", BF16)
            got += sp.sp24_gemm_fp8_fused(*w8, M, c, s, bias, "silu", r, True)
        return got

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = run()
    for k in range(3):
        for i, (x, (c, s), r) in enumerate(zip(xs, q8, rs)):
            x.copy_(rand(10 * k + i, *x.shape))
            nc, ns = sp.sp24_quant_fp8(x)
            c.copy_(nc), s.view(torch.uint8).copy_(ns.view(torch.uint8))
            r.copy_(rand(100 * k + i, *r.shape))
        bias.copy_(rand(50 + k, M))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(static, run()):
            assert torch.equal(a, b)


def test_products_on_another_stream():
    say("fused product on a side stream")
    M, K, N = 512, 256, 300
    values, meta = weight(1, M, K)
    side = torch.cuda.Stream()
    x = rand(2, N, K, dtype=BF16)
    want = sp.sp24_gemm_bf16_fused(values, meta, M, x, activation="gelu", layout="token")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            big = big @ big * 1e-3
        late = x.clone() + (big[0, 0] * 0).to(BF16).nan_to_num()
        got = sp.sp24_gemm_bf16_fused(values, meta, M, late, activation="gelu", layout="token")
    side.synchronize()
    assert torch.equal(got, want)


def test_products_refuse():
    say("fused products refuse")
    M, K, N = 64, 64, 8
    values, meta = weight(1, M, K)
    X, bias = rand(2, N, K, dtype=BF16), rand(3, M)
    call = lambda **kw: sp.sp24_gemm_bf16_fused(values, meta, M, X, **{"layout": "token", **kw})  # noqa: E731
    for bad in (dict(activation="tanh"), dict(bias=bias.to(BF16)), dict(bias=bias[:-1]), dict(bias=bias.cpu()), dict(residual=rand(4, N, M, dtype=BF16)),
                dict(residual=rand(4, M, N)), dict(residual=rand(4, N, 2 * M)[:, ::2]), dict(preact=rand(4, N, M, dtype=BF16)),
                dict(out=rand(4, N, M + 1)), dict(out_dtype=FP16), dict(layout="rows")):
        with pytest.raises(ValueError):
            call(**bad)
    Y, Z = rand(4, N, M), rand(5, N, M)
    for bad in (dict(out=Y, preact=Y), dict(residual=Z, preact=Z), dict(residual=rand(6, N, M + 1).flatten()[1:1 + N * M].view(N, M))):
        with pytest.raises(sp.Sp24Error):
            call(**bad)
    with pytest.raises(ValueError):
        sp.sp24_gemm_bf16_fused(values, meta, M + 16, X, layout="token")
    with pytest.raises(ValueError):
        sp.sp24_gemm_bf16_fused(values.cpu(), meta, M, X, layout="token")
