"""The epilogue's gradient against the formula in 64 bits and against differences of the activation.

dZ is one fp32 product of dY and the slope, rounded to dY's type: off by the slope's error and two roundings. dbias sums N
such products in fp32 in chains of at most N / 4 a thread and then 3 and 36 or fewer partial sums: within N U sum |dZ|."""
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import layer_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
SIZES = [(1, 1), (1, 8), (3, 5), (2, 768), (17, 513), (197, 768), (64, 1000), (300, 2047), (33, 28672), (5000, 16), (16, 512), (8200, 40), (1030, 4096)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def check(dZ, dbias, dY, Z, act):
    dy, z = dY.double(), Z.double()
    s = ref.slope(z, act)
    want = torch.where(z > 0, dy, 0.0) if act == "relu" else dy * s
    off32 = dy.abs() * ref.slope_error(z, act) + ref.U * want.abs()
    if dZ is not None:
        bound = off32 + (want.abs() + off32) * ref.UNIT[dY.dtype] * 1.0001 + (2.0 ** -25 if dY.dtype is torch.float16 else 1e-37)
        assert ((dZ.double() - want).abs() <= bound).all()
    if dbias is not None:
        near = off32.sum(0) + dy.shape[0] * ref.U * (want.abs() + off32).sum(0) + 1e-37
        assert ((dbias.double() - want.sum(0)).abs() <= near).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu", "relu", "silu"])
@pytest.mark.parametrize("N,M", SIZES)
def test_sizes(N, M, act, dtype):
    say(f"epilogue gradient {N}x{M} {act} {dtype}")
    dY, Z = rand(N, N, M, dtype=dtype), rand(M, N, M, dtype=dtype, scale=2.0)
    dZ, dbias = sp.sp24_epilogue_backward(dY, Z, act)
    check(dZ, dbias, dY, Z, act)
    again = sp.sp24_epilogue_backward(dY, Z, act)
    assert torch.equal(again[0], dZ) and torch.equal(again[1], dbias)
    only, none = sp.sp24_epilogue_backward(dY, Z, act, want_dbias=False)
    assert none is None and torch.equal(only, dZ)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,M", SIZES)
def test_bias_alone(N, M, dtype):
    say(f"bias gradient {N}x{M} {dtype}")
    dY = rand(N, N, M, dtype=dtype)
    dZ, dbias = sp.sp24_epilogue_backward(dY)
    assert dZ.data_ptr() == dY.data_ptr()
    near = N * ref.U * dY.double().abs().sum(0)
    assert ((dbias.double() - dY.double().sum(0)).abs() <= near).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pads", [(1, 2, 3), (8, 8, 8), (0, 5, 16)])
def test_pitches_and_in_place(dtype, pads):
    say(f"epilogue gradient pitches {dtype} {pads}")
    N, M = 100, 1029
    bufs = [torch.full((N, M + p), float("nan"), dtype=dtype, device="cuda") for p in pads]
    dY, Z, dZ = (b[:, :M] for b in bufs)
    dY.copy_(rand(1, N, M)), Z.copy_(rand(2, N, M))
    want = sp.sp24_epilogue_backward(dY.contiguous(), Z.contiguous(), "silu")
    got = sp.sp24_epilogue_backward(dY, Z, "silu", dZ=dZ)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for b in bufs:
        assert torch.isnan(b[:, M:]).all()
    for target in (dY, Z):
        y, z = (t.clone() if t is not target else t for t in (dY, Z))
        keep = target.clone()
        got = sp.sp24_epilogue_backward(y, z, "silu", dZ=target)
        assert torch.equal(target, want[0]) and torch.equal(got[1], want[1])
        target.copy_(keep)


@pytest.mark.parametrize("act", ["gelu", "relu", "silu"])
def test_against_differences(act):
    """Central differences of the activation in 64 bits: the error of a step h is h^2 / 6 of the third derivative (below 2)
    and 2^-53 / h; ReLU away from its corner."""
    say(f"epilogue gradient differences {act}")
    z = torch.linspace(-8, 8, 4096, device="cuda")
    z = z[z.abs() > 1e-3] if act == "relu" else z
    h = 1e-5
    d = (ref.act(z.double() + h, act) - ref.act(z.double() - h, act)) / (2 * h)
    dZ, _ = sp.sp24_epilogue_backward(torch.ones_like(z)[None], z[None], act)
    assert ((dZ[0].double() - d).abs() <= 20 * ref.U + 1e-9).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu", "relu", "silu"])
def test_special_values(act, dtype):
    """Infinite and NaN z: the slope's limits, and NaN; ReLU takes an infinite dY only where it passes."""
    say(f"epilogue gradient special values {act} {dtype}")
    inf, nan = float("inf"), float("nan")
    big = torch.finfo(dtype).max
    z = torch.tensor([[inf, -inf, big, -big, 0.0, -0.0, 100.0, -100.0, nan]], device="cuda").to(dtype)
    dY = torch.full_like(z, 2.0)
    dZ, dbias = sp.sp24_epilogue_backward(dY, z, act)
    want = torch.tensor([[2.0, 0.0, 2.0, 0.0, 0.0 if act == "relu" else 1.0, 0.0 if act == "relu" else 1.0, 2.0, 0.0, 0.0 if act == "relu" else nan]])
    assert torch.allclose(dZ.cpu().float(), want, rtol=0, atol=1e-6, equal_nan=True)
    assert torch.allclose(dbias.cpu(), want[0], rtol=0, atol=1e-6, equal_nan=True)
    if act == "relu":
        dZ, _ = sp.sp24_epilogue_backward(torch.full_like(z, inf), z, act)
        assert torch.equal(dZ.cpu().float(), torch.tensor([[inf, 0, inf, 0, 0, 0, inf, 0, 0]]))


def test_captured_and_replayed():
    say("epilogue gradient in a graph")
    dY, Z = rand(1, 700, 1000, dtype=torch.bfloat16), rand(2, 700, 1000, dtype=torch.bfloat16)
    sp.sp24_epilogue_backward(dY, Z, "gelu")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = sp.sp24_epilogue_backward(dY, Z, "gelu")
    for k in range(3):
        dY.copy_(rand(10 + k, 700, 1000)), Z.copy_(rand(20 + k, 700, 1000))
        graph.replay()
        torch.cuda.synchronize()
        want = sp.sp24_epilogue_backward(dY, Z, "gelu")
        assert torch.equal(static[0], want[0]) and torch.equal(static[1], want[1])


def test_refusals():
    say("epilogue gradient refuses")
    dY, Z = rand(1, 4, 16), rand(2, 4, 16)
    for args, kw in (((dY,), dict(activation="gelu")), ((dY, Z), {}), ((dY, Z.half(), "gelu"), {}), ((dY, Z[:3], "gelu"), {}), ((dY, Z, "tanh"), {}),
                     ((dY, Z.cpu(), "gelu"), {}), ((dY.cpu(), Z, "gelu"), {}), ((dY.int(), Z, "gelu"), {}), ((dY,), dict(dZ=Z)),
                     ((dY, Z, "gelu"), dict(dbias=Z[0].half())), ((dY.t().contiguous().t(), Z, "gelu"), {})):
        with pytest.raises(ValueError):
            sp.sp24_epilogue_backward(*args, **kw)
    with pytest.raises(sp.Sp24Error):  # the base is not on 16 bytes
        sp.sp24_epilogue_backward(rand(3, 65)[1:].view(4, 16), Z, "gelu")
