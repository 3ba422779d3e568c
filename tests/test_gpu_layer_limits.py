"""The layer operators at the ends of what they accept."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests.gpu_util import require_gpu, say
from tests.test_gpu_layer_adamw import HYPER, check, expect, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_least_eps(bits):
    """With the least eps a weight without gradient stays zero, the others move by their formula."""
    say(f"adamw least eps, {bits} bits")
    hyper = {**HYPER, "eps": 2.0 ** -126}
    p, g = rand(1, 3000), rand(2, 3000)
    p[::3], g[::3] = 0, 0
    state = sp.sp24_adamw_state(p, bits)
    with np.errstate(invalid="ignore", divide="ignore"):
        for step in (1, 2, 3):
            want = expect(p, g, state, step, seed=5, **hyper)
            sp.sp24_adamw([p], [g], [state], step, seed=5, **hyper)
            check(p, state, *want)
            assert (p[::3] == 0).all() and torch.isfinite(p).all()
    for eps in (1e-39, 0.0):
        with pytest.raises(sp.Sp24Error):
            sp.sp24_adamw([p], [g], [state], 4, **{**hyper, "eps": eps})


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("later", [False, True])
@pytest.mark.parametrize("lr,decay", [(3.4e38, 0.0), (1e10, 3e38), (3e38, 3e38)])
def test_adamw_rates_past_fp32(bits, later, lr, decay):
    """Where lr / (1 - beta1^t) or lr weight_decay pass fp32 a weight that has nothing to change stays zero."""
    say(f"adamw rates past fp32, {bits} bits, lr {lr}, decay {decay}, on the device {later}")
    p, g = torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda")
    p[500:], g[500:] = 1.0, 1.0
    state = sp.sp24_adamw_state(p, bits)
    rate = torch.tensor(lr, device="cuda") if later else lr
    sp.sp24_adamw([p], [g], [state], 1, lr=rate, weight_decay=decay)
    assert (p[:500] == 0).all() and not (p[500:] == 1).any()


def test_adamw_groups_round_independently():
    """Two calls, each with its parameters' places in the model, are one call over all of them; without, equal parameters would
    share their random bits from call to call."""
    say("adamw groups")
    g = [rand(1, 5000)] * 4 + [rand(2, 300)]
    p = [torch.zeros_like(x) for x in g]
    one, two = ([sp.sp24_adamw_state(x, 8) for x in p] for _ in range(2))
    sp.sp24_adamw(p, g, one, 1, seed=3, first_index=7)
    at = 2
    sp.sp24_adamw(p[:at], g[:at], two[:at], 1, seed=3, first_index=7)
    sp.sp24_adamw(p[at:], g[at:], two[at:], 1, seed=3, first_index=7 + at)
    for a, b in zip(one, two):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    for i in range(4):
        for j in range(i):
            assert not torch.equal(one[i][0].view(torch.uint8), one[j][0].view(torch.uint8))
    want = expect(torch.zeros(300, device="cuda"), g[4], sp.sp24_adamw_state(p[4], 8), 1, index=11, seed=3, lr=1e-3, weight_decay=0.01)
    check(p[4], two[4], want[0], np.full(300, np.inf), want[2])  # the state; two calls moved the weight
    last = [torch.zeros(8, device="cuda")]
    sp.sp24_adamw(last, last, [sp.sp24_adamw_state(last[0], 8)], 1, first_index=2 ** 32 - 1)


def test_adamw_refuses_tensors_in_two_roles():
    """Scales that two moments share, and outputs that another tensor still reads: which comes first would be left to chance."""
    say("adamw refuses tensors in two roles")
    p, g = [rand(i, 256) for i in range(2)], [rand(9, 256)] * 2
    for bits in (32, 8):
        s = [sp.sp24_adamw_state(x, bits) for x in p]
        t = [sp.sp24_adamw_state(x, bits) for x in p]
        q = [torch.empty_like(x) for x in p]
        for out in ((p[::-1], s), (p, s[::-1]), ([p[1], q[0]], t), (q, [s[1], t[0]]), (q, [(t[0][0], *s[1][1:]), t[1]])):
            with pytest.raises(ValueError):
                sp.sp24_adamw(p, g, s, 1, out=out)
        if bits == 8:
            with pytest.raises(ValueError):
                sp.sp24_adamw(p, g, [(s[0][0], s[0][1], s[0][2], s[0][1]), s[1]], 1)
            with pytest.raises(ValueError):
                sp.sp24_adamw(p, g, [s[0], (s[1][0], s[0][1], s[1][2], s[1][3])], 1)
        before = [x.clone() for x in p]
        sp.sp24_adamw(p, g, s, 1, out=(q, t))  # elsewhere, in place, and some of each
        sp.sp24_adamw(p, g, s, 1, out=([p[0], q[1]], [t[0], s[1]]))
        assert torch.equal(p[0], q[0]) and torch.equal(p[1], before[1]) and not torch.equal(q[1], p[1])
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(s[1], t[1]))


def strided(batch, rows, cols, dtype, fill=float("nan")):
    """(buffer, its entries of rows x cols whose strides are the least multiples of 16 bytes, plus 16)."""
    unit = 16 // dtype.itemsize
    entry = (-(-rows * cols // unit) + 1) * unit
    buf = torch.full((batch, entry), fill, dtype=dtype, device="cuda")
    return buf, buf.as_strided((batch, rows, cols), (entry, cols, 1))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout,M,K,N", [("token", 70, 64, 30), ("token", 7, 128, 1), ("token", 33, 64, 131), ("feature", 30, 64, 70), ("feature", 257, 128, 129), ("feature", 9, 48, 5)])
def test_batched_entries_of_odd_sizes(layout, M, K, N, out):
    """Entries that are no multiple of 16 bytes, in outputs and residuals of padded strides: each as by itself, nothing beside it written."""
    say(f"bf16 fused batch of odd entries {layout} {M}x{K} N={N} {out}")
    values, meta = sp.sp24_prune_compress(rand(1, M, K, dtype=torch.bfloat16))
    X = rand(2, 3, *((N, K) if layout == "token" else (K, N)), dtype=torch.bfloat16)
    if layout == "feature":  # X's entries lie on 16 bytes too
        x = strided(3, K, N, torch.bfloat16)[1]
        X = x.copy_(X)
    bias, shape = rand(3, M), ((N, M) if layout == "token" else (M, N))
    ybuf, Y = strided(3, *shape, out)
    zbuf, Z = strided(3, *shape, out)
    _, R = strided(3, *shape, out)
    R.copy_(rand(4, 3, *shape))
    how = dict(bias=bias, activation="silu", layout=layout, out_dtype=out)
    got = sp.sp24_gemm_bf16_fused(values, meta, M, X, residual=R, preact=Z, out=Y, **how)
    assert got[0].data_ptr() == Y.data_ptr() and got[1].data_ptr() == Z.data_ptr()
    for b in range(3):
        one = sp.sp24_gemm_bf16_fused(values, meta, M, X[b].contiguous(), residual=R[b].contiguous(), preact=True, **how)
        assert torch.equal(Y[b], one[0]) and torch.equal(Z[b], one[1])
    for buf in (ybuf, zbuf):
        assert torch.isnan(buf[:, shape[0] * shape[1]:]).all()
    inplace = strided(3, *shape, out)[1].copy_(R)
    sp.sp24_gemm_bf16_fused(values, meta, M, X, residual=inplace, out=inplace, **how)
    assert torch.equal(inplace, Y)


@pytest.mark.parametrize("act", ["gelu", "relu", "silu"])
def test_feature_major_gradient_without_bias(act):
    """dZ of a feature-major Z is the token-major one's transpose."""
    say(f"feature-major epilogue gradient {act}")
    for dtype in (torch.bfloat16, torch.float32):
        dY, Z = rand(1, 130, 196, dtype=dtype), rand(2, 130, 196, dtype=dtype)
        dZ, none = sp.sp24_epilogue_backward(dY, Z, act, want_dbias=False)
        want, _ = sp.sp24_epilogue_backward(dY.t().contiguous(), Z.t().contiguous(), act)
        assert none is None and torch.equal(dZ, want.t())
