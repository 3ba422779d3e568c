"""Host-side checks of the 8-bit floating-point entry points (no GPU, no kernel launched): invalid arguments are
rejected before any HIP call, sizes, and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import fp8_ref as ref
from tests.test_abi import A, B, C, MIS, lib  # noqa: F401

BF16, FP16, FP32, I8, FP8 = sp.SP24_BF16, sp.SP24_FP16, sp.SP24_FP32, sp.SP24_I8, sp.SP24_FP8
NULL, SHAPE, ALIGN, DTYPE, ARG = (sp.SP24_ERR_NULL, sp.SP24_ERR_SHAPE, sp.SP24_ERR_ALIGN, sp.SP24_ERR_DTYPE,
                                  sp.SP24_ERR_ARG)
D = ctypes.c_void_p(0x40000)
E = ctypes.c_void_p(0x50000)
ODD = ctypes.c_void_p(0x10001)


def changed(good, **kw):
    """The valid arguments `good` (a dict in order) with some of them replaced."""
    assert set(kw) <= set(good)
    return tuple({**good, **kw}.values())


QUANT = dict(X=A, dtype=BF16, N=2, K=48, ldx=48, codes=B, ldc=48, scales=C, lds=1, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(X=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(dtype=I8), DTYPE),
    (dict(dtype=FP8), DTYPE), (dict(dtype=-1), DTYPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(K=40), SHAPE), (dict(ldx=32), SHAPE),
    (dict(ldc=32), SHAPE), (dict(lds=0), SHAPE), (dict(K=144, ldx=144, ldc=144, lds=1), SHAPE),
    (dict(K=1 << 21, ldx=1 << 21, ldc=1 << 21, lds=1 << 14), SHAPE), (dict(ldx=1 << 23), SHAPE), (dict(lds=1 << 22), SHAPE),
    (dict(N=1 << 31), SHAPE),
    (dict(X=MIS), ALIGN), (dict(codes=MIS), ALIGN), (dict(ldx=52), ALIGN), (dict(ldc=56), ALIGN),
])
def test_quant_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_quant_fp8(*changed(QUANT, **bad)) == expect


NORM = dict(X=A, dtype=BF16, N=2, K=48, ldx=48, R=B, ldr=48, gamma=C, eps=1e-6, H=D, ldh=48, codes=E, ldc=48, scales=E,
            lds=1, rstd=None, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(X=None), NULL), (dict(gamma=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(H=None), NULL),
    (dict(R=None), ARG), (dict(dtype=I8), DTYPE), (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(N=0), SHAPE), (dict(K=56), SHAPE), (dict(ldx=32), SHAPE), (dict(ldr=32), SHAPE),
    (dict(ldh=32), SHAPE), (dict(ldc=32), SHAPE), (dict(lds=0), SHAPE), (dict(X=MIS), ALIGN), (dict(R=MIS), ALIGN),
    (dict(H=MIS), ALIGN), (dict(gamma=MIS), ALIGN), (dict(codes=MIS), ALIGN), (dict(ldr=52), ALIGN), (dict(rstd=ODD), ALIGN),
    (dict(K=32784, ldx=32784, ldr=32784, ldh=32784, ldc=32784, lds=257), SHAPE),
])
def test_rmsnorm_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_rmsnorm_fp8(*changed(NORM, **bad)) == expect


BACK = dict(dY=A, dtype=BF16, N=2, K=48, lddy=48, H=B, ldh=48, rstd=C, gamma=C, dH=D, lddh=48, dX=E, lddx=48, dgamma=E,
            workspace=E, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dY=None), NULL), (dict(H=None), NULL), (dict(rstd=None), NULL), (dict(gamma=None), NULL), (dict(dX=None), NULL),
    (dict(dgamma=None), NULL), (dict(workspace=None), NULL), (dict(dtype=I8), DTYPE), (dict(N=0), SHAPE), (dict(K=8), SHAPE),
    (dict(lddy=32), SHAPE), (dict(ldh=32), SHAPE), (dict(lddh=32), SHAPE), (dict(lddx=32), SHAPE), (dict(dY=MIS), ALIGN),
    (dict(H=MIS), ALIGN), (dict(dH=MIS), ALIGN), (dict(dX=MIS), ALIGN), (dict(workspace=MIS), ALIGN), (dict(rstd=ODD), ALIGN),
    (dict(dgamma=ODD), ALIGN), (dict(lddx=52), ALIGN),
])
def test_rmsnorm_backward_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_rmsnorm_backward(*changed(BACK, **bad)) == expect


PRUNE = dict(W=A, dtype=BF16, M=4, K=48, ldw=48, score=0, norms=None, values=B, meta=C, w_scales=D, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(W=None), NULL), (dict(values=None), NULL), (dict(meta=None), NULL), (dict(w_scales=None), NULL),
    (dict(score=1), NULL), (dict(norms=A), ARG), (dict(score=2), ARG), (dict(dtype=I8), DTYPE), (dict(M=0), SHAPE),
    (dict(K=24), SHAPE), (dict(ldw=32), SHAPE), (dict(W=MIS), ALIGN), (dict(values=MIS), ALIGN), (dict(meta=MIS), ALIGN),
    (dict(score=1, norms=MIS), ALIGN), (dict(ldw=52), ALIGN), (dict(M=(1 << 22) + 1), SHAPE),
    (dict(M=1 << 22, K=1 << 20, ldw=1 << 20), SHAPE),
])
def test_prune_compress_fp8_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_prune_compress_fp8(*changed(PRUNE, **bad)) == expect


UNPRUNE = dict(values=A, meta=B, w_scales=C, M=4, K=48, W_out=D, out_dtype=BF16, ldw=48, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(values=None), NULL), (dict(W_out=None), NULL), (dict(out_dtype=FP16), DTYPE), (dict(M=0), SHAPE), (dict(K=8), SHAPE),
    (dict(ldw=32), SHAPE), (dict(W_out=MIS), ALIGN), (dict(values=MIS), ALIGN), (dict(ldw=52), ALIGN),
])
def test_decompress_fp8_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_decompress_fp8(*changed(UNPRUNE, **bad)) == expect


GEMM = dict(values=A, meta=B, w_scales=C, M=4, K=48, X=D, N=2, ldx=48, x_scales=C, lds=1, Y=E, out_dtype=BF16, ldy=4, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(values=None), NULL), (dict(meta=None), NULL), (dict(w_scales=None), NULL), (dict(X=None), NULL),
    (dict(x_scales=None), NULL), (dict(Y=None), NULL), (dict(out_dtype=FP32), DTYPE), (dict(out_dtype=FP8), DTYPE),
    (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=40), SHAPE), (dict(ldx=32), SHAPE), (dict(lds=0), SHAPE), (dict(ldy=3), SHAPE),
    (dict(X=MIS), ALIGN), (dict(Y=MIS), ALIGN), (dict(values=MIS), ALIGN), (dict(meta=MIS), ALIGN), (dict(ldx=56), ALIGN),
    (dict(M=(1 << 22) + 1, ldy=(1 << 22) + 1), SHAPE), (dict(M=1 << 22, ldy=1 << 22, N=1 << 30), SHAPE),
])
def test_gemm_fp8_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_gemm_fp8(*changed(GEMM, **bad)) == expect


GRAD = dict(dY=A, N=2, M=8, lddy=8, X=B, K=48, ldx=48, x_scales=C, lds=1, meta=D, dW=E, out_dtype=BF16, ldw=48,
            workspace=None, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dY=None), NULL), (dict(X=None), NULL), (dict(x_scales=None), NULL), (dict(dW=None), NULL), (dict(out_dtype=FP16), DTYPE),
    (dict(N=0), SHAPE), (dict(M=0), SHAPE), (dict(K=8), SHAPE), (dict(lddy=7), SHAPE), (dict(ldx=32), SHAPE), (dict(lds=0), SHAPE),
    (dict(ldw=32), SHAPE), (dict(dY=MIS), ALIGN), (dict(X=MIS), ALIGN), (dict(dW=MIS), ALIGN), (dict(meta=MIS), ALIGN),
    (dict(lddy=12), ALIGN), (dict(ldw=52), ALIGN), (dict(workspace=MIS), ALIGN),
    (dict(N=8192), NULL),  # many tokens, few tiles: needs its workspace
])
def test_grad_weight_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_grad_weight_fp8(*changed(GRAD, **bad)) == expect


def test_sizes(lib):  # noqa: F811
    assert sp.sp24_compressed_bytes(17, 144, torch.float8_e4m3fn) == sp.sp24_compressed_bytes(17, 144, torch.int8)
    n = ctypes.c_int64(-1)
    for bad in ((0, 48), (4, 40), (4, 32784)):
        assert lib.sp24_rmsnorm_backward_bytes(*bad, ctypes.byref(n)) == SHAPE
    assert lib.sp24_rmsnorm_backward_bytes(1, 48, ctypes.byref(n)) == 0 and n.value >= 48 * 4
    assert lib.sp24_rmsnorm_backward_bytes(1, 48, None) == NULL
    assert lib.sp24_grad_weight_fp8_bytes(8, 48, 2, None) == NULL
    assert lib.sp24_grad_weight_fp8_bytes(0, 48, 2, ctypes.byref(n)) == SHAPE
    assert lib.sp24_grad_weight_fp8_bytes(8, 48, 2, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.sp24_grad_weight_fp8_bytes(8, 48, 8192, ctypes.byref(n)) == 0 and n.value >= 2 * 8 * 48 * 4


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 48, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sp.sp24_quant_fp8(x)
    with pytest.raises(ValueError):
        sp.sp24_rmsnorm_fp8(x, x[0])


def test_plain_codes():
    """The plain rounding against every e4m3 number, its neighbours' midpoints, and torch's conversion."""
    every = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(every), every) and np.array_equal(ref.e4m3(-every), -every)
    mid = (every[1:] + every[:-1]) / 2  # ties: to the neighbour with the even code
    assert np.array_equal(ref.e4m3(mid), np.where(np.arange(126) % 2 == 0, every[:-1], every[1:]))
    v = np.random.default_rng(0).uniform(-448, 448, 10000).astype(np.float32)
    assert np.array_equal(ref.e4m3(v.astype(np.float64)), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())
    assert list(ref.scale_exp(np.array([0.0, 448.0, 448.001, 224.0, 224.001, 1e-45]))) == [-127, 0, 1, -1, 0, -127]


def test_binding_takes_keywords():
    """Every operand can be given by its name, the first one too (host tensors: refused as such, not as a wrong call)."""
    x = torch.zeros(16, 128, dtype=torch.bfloat16)
    codes, scales = x.to(torch.float8_e4m3fn), torch.zeros(16, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    values, meta, w_scales = torch.zeros(1024).to(torch.float8_e4m3fn), torch.zeros(256, dtype=torch.uint8), scales[:1]
    for call in (lambda: sp.sp24_prune_compress_fp8(W=x), lambda: sp.sp24_decompress_fp8(values=values, meta=meta, w_scales=w_scales, M=16, K=128),
                 lambda: sp.sp24_decompress_fp8(M=16, K=128, w_scales=w_scales, meta=meta, values=values), lambda: sp.sp24_quant_fp8(X=x),
                 lambda: sp.sp24_rmsnorm_fp8(X=x, gamma=x[0]), lambda: sp.sp24_rmsnorm_backward(dY=x, H=x, rstd=x[:, 0].float(), gamma=x[0]),
                 lambda: sp.sp24_gemm_fp8(values=values, meta=meta, w_scales=w_scales, M=16, X=codes, x_scales=scales),
                 lambda: sp.sp24_grad_weight_fp8(dY=x, X=codes, x_scales=scales)):
        with pytest.raises(ValueError, match="device tensors only"):
            call()


def test_launch_limits(lib):  # noqa: F811
    """What would need 2^32 threads or more in one launch is a shape error before any HIP call."""
    wide = dict(M=1 << 22, K=16, ldx=16, ldy=1 << 22)
    # 2^14 tile rows x 512 tiles of 256 tokens, 512 threads each: 2^32
    assert lib.sp24_gemm_fp8(*changed(GEMM, **wide, N=511 * 256 + 1)) == SHAPE
    n = ctypes.c_int64(-1)
    # 2^14 x 2^9 and 2^14 x 2^12 tiles of 256 x 256, 512 threads each: 2^32 and 2^35
    for K in (511 * 256 + 16, 1 << 20):
        assert lib.sp24_grad_weight_fp8_bytes(1 << 22, K, 64, ctypes.byref(n)) == SHAPE
        assert lib.sp24_grad_weight_fp8(*changed(GRAD, N=64, M=1 << 22, lddy=1 << 22, K=K, ldx=K, lds=1 << 13, ldw=K)) == SHAPE
    assert lib.sp24_grad_weight_fp8_bytes(1 << 22, 511 * 256, 64, ctypes.byref(n)) == 0 and n.value == 0


@pytest.mark.parametrize("M,K", [(128, 128), (640, 640), (768, 768), (2048, 1024)])
def test_no_part_without_tokens(lib, M, K):  # noqa: F811
    """The tokens' parts of the weight's gradient, 128 tokens at a time: as many partial sums as parts that hold some."""
    n = ctypes.c_int64(-1)
    for N in (512, 600, 1000, 1300, 2000, 2049, 3000, 5000, 6304, 20000):
        assert lib.sp24_grad_weight_fp8_bytes(M, K, N, ctypes.byref(n)) == 0 and n.value % (4 * M * K) == 0
        parts = n.value // (4 * M * K)
        if parts:
            steps = -(-N // 128)
            assert parts > 1 and parts == -(-steps // -(-steps // parts))
