"""Host-side checks of the layer entry points (no GPU, no kernel launched): invalid arguments are rejected before any HIP
call, sizes, and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import layer_ref as ref
from tests.test_abi import A, B, C, MIS, lib  # noqa: F401
from tests.test_fp8_host import ALIGN, ARG, D, DTYPE, E, NULL, ODD, SHAPE, changed

BF16, FP16, FP32, I8, FP8 = sp.SP24_BF16, sp.SP24_FP16, sp.SP24_FP32, sp.SP24_I8, sp.SP24_FP8
GELU = sp.SP24_ACT_GELU
F, G = ctypes.c_void_p(0x60000), ctypes.c_void_p(0x70000)

BF16_FUSED = dict(values=A, meta=B, M=32, K=64, X=C, N=8, ldx=64, sx=512, bias=F, act=GELU, R=D, ldr=32, sr=256, Z=E, ldz=32, sz=256,
                  Y=G, out=FP32, ldy=32, sy=256, batch=1, layout=sp.SP24_TOKEN_MAJOR, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(values=None), NULL), (dict(meta=None), NULL), (dict(X=None), NULL), (dict(Y=None), NULL), (dict(out=FP16), DTYPE), (dict(out=I8), DTYPE),
    (dict(act=4), ARG), (dict(act=-1), ARG), (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=40), SHAPE), (dict(ldx=63), SHAPE), (dict(ldy=31), SHAPE),
    (dict(ldr=31), SHAPE), (dict(ldz=31), SHAPE), (dict(R=MIS), ALIGN), (dict(Z=MIS), ALIGN), (dict(Y=MIS), ALIGN), (dict(bias=ODD), ALIGN),
    (dict(Z=G), ARG), (dict(Z=D), ARG), (dict(R=G, ldr=40), ARG), (dict(layout=2), ARG), (dict(batch=0), SHAPE),
    (dict(batch=2, sr=-16), SHAPE), (dict(batch=2, sz=252), SHAPE), (dict(batch=2, sy=252), SHAPE), (dict(batch=2, sr=258), ALIGN),
    (dict(batch=2, sz=258), ALIGN), (dict(batch=2, R=G, sr=512), ARG),
])
def test_bf16_fused_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_gemm_bf16_fused(*changed(BF16_FUSED, **bad)) == expect


FP8_FUSED = dict(values=A, meta=B, ws=B, M=32, K=144, X=C, N=8, ldx=144, xs=D, lds=2, bias=F, act=GELU, R=D, ldr=32, Z=E, ldz=32, Y=G, out=BF16,
                 ldy=32, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(values=None), NULL), (dict(meta=None), NULL), (dict(ws=None), NULL), (dict(X=None), NULL), (dict(xs=None), NULL), (dict(Y=None), NULL),
    (dict(out=FP32), DTYPE), (dict(act=4), ARG), (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=136), SHAPE), (dict(ldx=128), SHAPE),
    (dict(lds=1), SHAPE), (dict(ldy=31), SHAPE), (dict(ldr=31), SHAPE), (dict(ldz=31), SHAPE), (dict(ldr=1 << 23), SHAPE), (dict(ldz=1 << 23), SHAPE),
    (dict(R=MIS), ALIGN), (dict(Z=MIS), ALIGN), (dict(Y=MIS), ALIGN), (dict(bias=ODD), ALIGN), (dict(Z=G), ARG), (dict(Z=D), ARG),
    (dict(R=G, ldr=40), ARG),
])
def test_fp8_fused_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_gemm_fp8_fused(*changed(FP8_FUSED, **bad)) == expect


BACK = dict(dY=A, dtype=BF16, N=100, M=33, lddy=33, Z=B, ldz=33, act=GELU, dZ=C, lddz=33, dbias=D, workspace=E, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dY=None), NULL), (dict(Z=None), NULL), (dict(dZ=None), NULL), (dict(N=1000, workspace=None), NULL), (dict(dtype=I8), DTYPE), (dict(act=7), ARG),
    (dict(act=0), ARG), (dict(act=0, Z=None), ARG), (dict(act=0, Z=None, dZ=None, dbias=None), NULL), (dict(N=0), SHAPE), (dict(M=0), SHAPE),
    (dict(N=1 << 31), SHAPE), (dict(M=(1 << 22) + 1, lddy=1 << 23, ldz=1 << 23, lddz=1 << 23), SHAPE), (dict(lddy=32), SHAPE), (dict(ldz=32), SHAPE),
    (dict(lddz=32), SHAPE), (dict(lddy=1 << 23), SHAPE), (dict(dY=MIS), ALIGN), (dict(Z=MIS), ALIGN), (dict(dZ=MIS), ALIGN),
    (dict(workspace=MIS), ALIGN), (dict(dbias=ODD), ALIGN), (dict(dZ=A, lddz=40), ARG), (dict(dZ=B, lddz=40), ARG),
])
def test_epilogue_backward_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_epilogue_backward(*changed(BACK, **bad)) == expect


def test_epilogue_backward_bytes(lib):  # noqa: F811
    n = ctypes.c_int64()
    assert lib.sp24_epilogue_backward_bytes(0, 8, ctypes.byref(n)) == SHAPE and lib.sp24_epilogue_backward_bytes(8, 8, None) == NULL
    assert lib.sp24_epilogue_backward_bytes(1, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.sp24_epilogue_backward_bytes(8192, 28672, ctypes.byref(n)) == 0 and n.value > 0 and n.value % (4 * 28672) == 0


class Tensor(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("p", "p_out", "g", "m", "m_out", "v", "v_out", "ms", "ms_out", "vs", "vs_out", "copy")] + \
               [("n", ctypes.c_int64), ("index", ctypes.c_int64)]


T32 = dict(p=0x10000, p_out=0x10000, g=0x20000, m=0x30000, m_out=0x30000, v=0x40000, v_out=0x40000, ms=None, ms_out=None, vs=None, vs_out=None,
           copy=0x50000, n=100, index=0)
T8 = {**T32, "ms": 0x60001, "ms_out": 0x60001, "vs": 0x70001, "vs_out": 0x70001}
ADAM = dict(count=1, grad=BF16, state=FP32, copy=BF16, lr=1e-3, lr_dev=None, step=1, step_dev=None, b1=0.9, b2=0.999, eps=1e-8, decay=0.1,
            scale=None, seed=0, workspace=None, stream=None)


@pytest.mark.parametrize("bad,expect", [
    (dict(count=-1), SHAPE), (dict(grad=I8), DTYPE), (dict(state=BF16), DTYPE), (dict(copy=FP32), DTYPE), (dict(lr=-1.0), ARG), (dict(lr=float("inf")), ARG),
    (dict(lr=float("nan")), ARG), (dict(step=0), ARG), (dict(b1=1.0), ARG), (dict(b1=-0.1), ARG), (dict(b2=1.0), ARG), (dict(b2=float("nan")), ARG),
    (dict(eps=0.0), ARG), (dict(eps=1e-60), ARG), (dict(eps=float("nan")), ARG), (dict(decay=-0.1), ARG), (dict(workspace=A), ARG), (dict(step_dev=A), NULL), (dict(lr_dev=A), NULL),
    (dict(lr_dev=A, workspace=MIS), ALIGN), (dict(lr_dev=ODD, workspace=A), ALIGN), (dict(step_dev=ctypes.c_void_p(0x10004), workspace=A), ALIGN), (dict(scale=ODD), ALIGN),
])
def test_adamw_validation(lib, bad, expect):  # noqa: F811
    assert lib.sp24_adamw((Tensor * 1)(Tensor(**T32)), *changed(ADAM, **bad)) == expect
    assert lib.sp24_adamw(None, *changed(ADAM)) == NULL


@pytest.mark.parametrize("state,bad,expect", [
    (FP32, dict(n=-1), SHAPE), (FP32, dict(n=(1 << 34) + 1), SHAPE), (FP32, dict(index=-1), ARG), (FP32, dict(index=1 << 32), ARG), (FP32, dict(ms=0x60000), ARG),
    *[(FP32, {k: None}, NULL) for k in ("p", "p_out", "g", "m", "m_out", "v", "v_out")],
    *[(FP8, {k: None}, NULL) for k in ("ms", "ms_out", "vs", "vs_out")],
    *[(FP32, {k: 0x10008 * 16 + 8}, ALIGN) for k in ("p", "p_out", "g", "m", "m_out", "v", "v_out", "copy")],
    # outputs that overlap their input without being it
    (FP32, dict(p_out=0x10010), ARG), (FP32, dict(m_out=0x30000 - 0x10), ARG), (FP32, dict(v_out=0x40000 + 0x180), ARG), (FP8, dict(m_out=0x30040), ARG),
    (FP8, dict(n=1000, ms_out=0x60004), ARG), (FP8, dict(n=1000, vs_out=0x70000), ARG),
])
def test_adamw_tensor_validation(lib, state, bad, expect):  # noqa: F811
    good = T8 if state == FP8 else T32
    both = (Tensor * 2)(Tensor(**good), Tensor(**{**good, **bad}))
    assert lib.sp24_adamw(both, *changed(ADAM, count=2, state=state)) == expect


def test_cpu_tensors_are_refused():
    x = torch.zeros(8, 64)
    with pytest.raises(ValueError):
        sp.sp24_adamw([x], [x], [sp.sp24_adamw_state(x)], 1)
    with pytest.raises(ValueError):
        sp.sp24_epilogue_backward(x)
    with pytest.raises(ValueError):
        sp.sp24_gemm_bf16_fused(x, x, 8, x.bfloat16(), layout="token")
    with pytest.raises(ValueError):
        sp.sp24_gemm_fp8_fused(x, x, x, 8, x.to(torch.float8_e4m3fn), x)
    with pytest.raises(ValueError):
        sp.sp24_gemm_bf16_fused(x, x, 8, x.bfloat16(), activation="tanh")


def test_zero_states():
    for n in (0, 1, 128, 129):
        p = torch.zeros(n)
        assert [t.numel() for t in sp.sp24_adamw_state(p)] == [n, n]
        assert [t.numel() for t in sp.sp24_adamw_state(p, 8)] == [n, -(-n // 128)] * 2


# ---------------------------------------------------------------- the plain forms themselves

def test_plain_codes_bracket_their_values():
    """A code stands for a neighbour of its value, the nearer end more often: mean of all 2^16 roundings within 2^-16 of a step."""
    r = np.arange(1 << 16)
    for x in (1.0, 3.3, 447.9, 0.001, 2.0 ** -9 * 1.5, 100.0):
        m = np.full(1 << 16, x, np.float32)
        m[0] = 448.0
        codes, scales = ref.first_codes(m, r)
        got = ref.first_values(codes, scales)[128:]
        assert (scales == 127)[0] and set(np.unique(got)) <= {got.min(), got.max()} and got.min() <= np.float32(x) <= got.max()
        whole = np.full(128 * 512, x, np.float32)
        whole[::128] = 448.0
        codes, scales = ref.first_codes(whole, (np.arange(whole.size) // 128 * 128) % 65536)
        step = max(x / 8, 2.0 ** -9)
        assert abs(ref.first_values(codes, scales).reshape(-1, 128)[:, 1:].mean() - x) < step / 200
    for x in (1e-4, 0.7, 65024.5, 17.0):
        v = np.full(128 * 512, x, np.float32)
        v[::128] = 65025.0
        codes, scales = ref.second_codes(v, (np.arange(v.size) // 128 * 128) % 65536)
        got = ref.second_values(codes, scales).reshape(-1, 128)[:, 1:]
        c = np.floor(np.sqrt(x))
        assert (scales == 127).all() and abs(got.mean() - max(x, 1.0)) <= (2 * c + 1) / 200


def test_random_words_are_spread():
    """Words of neighbouring elements, steps and tensors: every bit set in half of them (within 5 deviations), none alike."""
    w = np.concatenate([ref.random_words(s, t, i, 4096) for s in (0, 1, 1 << 40) for t in (1, 2) for i in (0, 1, 2)])
    bits = (w[:, None] >> np.arange(32, dtype=np.uint32)) & 1
    assert (np.abs(bits.mean(0) - 0.5) < 5 * 0.5 / w.size ** 0.5).all()
    a, b = ref.random_words(5, 1, 0, 65536), ref.random_words(5, 2, 0, 65536)
    for half in (lambda x: x & 0xFFFF, lambda x: x >> 16):
        assert abs(np.corrcoef(half(a).astype(float), half(b).astype(float))[0, 1]) < 5 / 256
        assert abs(np.corrcoef(half(a)[1:].astype(float), half(a)[:-1].astype(float))[0, 1]) < 5 / 256
        assert np.histogram(half(a), 64, (0, 65536))[0].std() < 2 * 32
