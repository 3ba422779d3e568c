"""The AdamW step. Moments are fp32 with one rounding a step, so 32-bit states, and the codes and scales of 8-bit ones, are
compared bit for bit with tests/layer_ref.py. Weights: in fp32 the product with the decay and its subtraction round to U of
p and of the result; the update lr m / den to 8 U of itself (a root and a reciprocal of one unit each in the last place, two
products, a sum, and the rounded rate and root of the bias corrections)."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests import layer_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
HYPER = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 127, 128, 129, 1000, 2047, 2048, 2049, 5003, 70001]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rand(seed, *shape, dtype=torch.float32, scale=1.0, spread=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda") * scale
    return (x * torch.exp(spread * torch.randn(*shape, generator=g, device="cuda"))).to(dtype)


def host(t):
    return t.detach().cpu().view(torch.uint8).numpy() if t.element_size() == 1 else t.detach().float().cpu().numpy()


def moments_of(state):
    if len(state) == 2:
        return host(state[0]).reshape(-1), host(state[1]).reshape(-1)
    mc, ms, vc, vs = (host(t) for t in state)
    return ref.first_values(mc, ms), ref.second_values(vc, vs)


def expect(p, g, state, step, index=0, seed=0, scale=1.0, lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1):
    """(new weights in 64 bits, how far they may be off, new state as arrays)."""
    m0, v0 = moments_of(state)
    m, v = ref.moments(m0, v0, host(g).reshape(-1), *betas, scale)
    p0 = host(p).reshape(-1)
    want = ref.weights(p0, m, v, step, lr, *betas, eps, weight_decay)
    update = np.abs(want - p0.astype(np.float64) * (1 - lr * weight_decay))
    off = ref.U * (2 * np.abs(p0) + 2 * np.abs(want) + 10 * update) + 1e-37
    if len(state) == 2:
        return want, off, (m, v)
    r = ref.random_words(seed, step, index, p0.size)
    return want, off, (*ref.first_codes(m, r & 0xFFFF), *ref.second_codes(v, r >> 16))


def check(p, state, want, off, new_state):
    assert (np.abs(host(p).reshape(-1) - want) <= off).all()
    for got, exp in zip(state, new_state):
        assert np.array_equal(host(got).reshape(-1), exp), np.flatnonzero(host(got).reshape(-1) != exp)[:8]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("copy", [None, torch.bfloat16, torch.float16])
def test_steps_over_sizes(bits, grad, copy):
    """Four steps from zero over tensors of many sizes at once, in place, each against the step's formula from what was there."""
    say(f"adamw {bits} bits, gradients {grad}, copies {copy}")
    p = [rand(n, n) for n in SIZES]
    states = [sp.sp24_adamw_state(x, bits) for x in p]
    copies = None if copy is None else [torch.empty_like(x, dtype=copy) for x in p]
    for step in range(1, 5):
        g = [rand(100 * step + n, n, dtype=grad, scale=1e-2, spread=1.0) for n in SIZES]
        want = [expect(*a, step=step, index=i, seed=77 + (5 << 40)) for i, a in enumerate(zip(p, g, states))]
        sp.sp24_adamw(p, g, states, step, copies=copies, seed=77 + (5 << 40), **HYPER)
        for x, s, w in zip(p, states, want):
            check(x, s, *w)
        if copies is not None:
            assert all(torch.equal(c, x.to(copy)) for c, x in zip(copies, p))


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_takes(bits):
    """100 tensors, empty ones among them, some without a gradient; the same written elsewhere; each its own random bits."""
    say(f"adamw 100 tensors, {bits} bits")
    sizes = [(37 * i) % 700 for i in range(100)]
    p = [rand(i, n) for i, n in enumerate(sizes)]
    g = [None if i % 9 == 4 else rand(1000 + i, n, scale=0.1) for i, n in enumerate(sizes)]
    states = [sp.sp24_adamw_state(x, bits) for x in p]
    want = [None if x is None else expect(a, x, s, step=3, index=i, seed=9) for i, (a, x, s) in enumerate(zip(p, g, states)) if sizes[i]]
    want = iter(want)
    before = [x.clone() for x in p]
    out = [torch.full_like(x, float("nan")) for x in p], [tuple(torch.empty_like(t) for t in s) for s in states]
    sp.sp24_adamw(p, g, states, 3, seed=9, out=out, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(p, before))
    assert all((t.view(torch.uint8) == 0).all() for s in states for t in s)
    sp.sp24_adamw(p, g, states, 3, seed=9, **HYPER)
    for i, n in enumerate(sizes):
        w = next(want) if n else None
        if g[i] is None:
            assert torch.equal(p[i], before[i]) and torch.isnan(out[0][i]).all()
        elif n:
            check(p[i], states[i], *w)
            assert torch.equal(out[0][i], p[i])
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out[1][i], states[i]))


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_are_left_alone(bits):
    """Tensors inside larger buffers: what lies behind their last element stays."""
    say(f"adamw surroundings, {bits} bits")
    for n in (1, 129, 2047, 4100):
        bufs = [torch.full((n + 64,), 7.0, device="cuda") for _ in range(4)]
        p, g = bufs[0][:n], rand(1, n)
        if bits == 32:
            state = bufs[1][:n], bufs[2][:n]
            state[0].zero_(), state[1].zero_()
        else:
            raw = [torch.full((k + 64,), 7, dtype=torch.uint8, device="cuda") for k in (n, (n + 127) // 128, n, (n + 127) // 128)]
            state = tuple(r[:-64].view(t) for r, t in zip(raw, (torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8, torch.float8_e8m0fnu)))
            for t in state:
                t.view(torch.uint8).zero_()
        copy = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        sp.sp24_adamw([p], [g], [state], 1, copies=[copy[:n]], **HYPER)
        torch.cuda.synchronize()
        assert (bufs[0][n:] == 7).all() and (copy[n:] == 7).all()
        rest = [b[n:] for b in bufs[1:3]] if bits == 32 else [r[-64:] for r in raw]
        assert all((r == 7).all() for r in rest)


def test_pruned_weights_stay_zero():
    say("adamw keeps a 2:4 pattern")
    W = sp.sp24_prune_mask(rand(1, 64, 256), 2)[1]
    kept = W != 0
    for bits in (32, 8):
        p, state = W.clone(), sp.sp24_adamw_state(W, bits)
        for step in range(1, 6):
            sp.sp24_adamw([p], [rand(step, 64, 256) * kept], [state], step, **HYPER)
        assert (p[~kept] == 0).all() and (p[kept] != W[kept]).all()
        assert (state[0].view(torch.uint8)[~kept] & 0x7F == 0).all() if bits == 8 else (state[0][~kept] == 0).all()


def test_rounding_is_right_on_average():
    """m and v over many seeds: the mean of n roundings, each within one step of the value, lies within 6 steps / (2 sqrt n)."""
    say("adamw rounding on average")
    n, seeds = 4096, 400
    p, g = torch.zeros(n, device="cuda"), rand(1, n, spread=0.5)
    big = 1 << 20
    m, v = np.zeros(n), np.zeros(n)
    for s in range(seeds):
        state = sp.sp24_adamw_state(p, 8)
        out = [torch.empty_like(p)], [tuple(torch.empty_like(t) for t in state)]
        sp.sp24_adamw([p], [g], [state], 1, seed=s * big + s, out=out, **HYPER)
        a, b = moments_of(out[1][0])
        m += a.astype(np.float64) / seeds
        v += b.astype(np.float64) / seeds
    wm, wv = ref.moments(np.zeros(n, np.float32), np.zeros(n, np.float32), host(g), 0.9, 0.999)
    sm, sv = 2.0 ** (ref.spread(host(out[1][0][1]).astype(float), n) - 127), 4.0 ** (ref.spread(host(out[1][0][3]).astype(float), n) - 127)
    step_m = np.maximum(np.abs(wm) / 8, sm * 2.0 ** -9)
    c = np.floor(np.sqrt(wv / sv))
    assert (np.abs(m - wm) <= 6 * step_m / (2 * seeds ** 0.5)).all()
    assert (np.abs(v - wv) <= 6 * (2 * c + 1) * sv / (2 * seeds ** 0.5))[c >= 1].all()


def test_extremes_of_8_bit_states():
    """Blocks of zeros, the smallest and largest numbers, one large among small ones; a block with an infinite or NaN gradient
    reads NaN from then on, its neighbours do not."""
    say("adamw 8-bit extremes")
    n = 128 * 8
    g = torch.zeros(n, device="cuda")
    g[128:256] = 1e-30
    g[256:384] = 1e18
    g[384], g[385:512] = 1.0, 1e-6
    g[512:640] = rand(1, 128)
    g[640:768], g[700] = rand(2, 128), float("inf")
    g[768:896], g[800] = rand(3, 128), float("nan")
    g[896:] = rand(4, 128)
    p = torch.zeros(n, device="cuda")
    state = sp.sp24_adamw_state(p, 8)
    fine = np.r_[0:640, 896:1024]
    want, off, codes = expect(p[torch.from_numpy(fine).cuda()], g[torch.from_numpy(fine).cuda()], sp.sp24_adamw_state(p[:768], 8), step=1, seed=3)
    sp.sp24_adamw([p], [g], [state], 1, seed=3, **HYPER)
    got = host(p)
    assert (np.abs(got[fine] - want) <= off).all()
    assert np.array_equal(host(state[1])[[0, 1, 2, 3, 4, 7]], codes[1]) and np.array_equal(host(state[3])[[0, 1, 2, 3, 4, 7]], codes[3])
    assert (host(state[1])[5:7] == 255).all() and (host(state[3])[5:7] == 255).all()
    assert np.isnan(got[700]) and np.isnan(got[800]) and np.isfinite(np.delete(got, [700, 800])).all()
    vc = host(state[2])
    assert (vc[385:512] == 1).all() and (vc[:128] == 0).all()  # above zero: one unit at least
    sp.sp24_adamw([p], [torch.zeros_like(g)], [state], 2, seed=3, **HYPER)
    assert np.isnan(host(p)[640:896]).all() and np.isfinite(host(p)[fine]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_and_graph(bits):
    """Step, rate and scale on the device give what host values give, and a captured step follows them from replay to replay."""
    say(f"adamw graph, {bits} bits")
    sizes = [300, 5000]
    a, b = ([rand(i, n) for i, n in enumerate(sizes)] for _ in range(2))
    sa, sb = ([sp.sp24_adamw_state(x, bits) for x in a] for _ in range(2))
    g = [rand(9, n) for n in sizes]
    step, lr, scale = torch.ones((), dtype=torch.int64, device="cuda"), torch.full((1,), 1e-2, device="cuda"), torch.full((1,), 0.5, device="cuda")
    hyper = {**HYPER, "lr": lr}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sp.sp24_adamw(b, g, sb, step, grad_scale=scale, seed=4, **hyper)
    torch.cuda.current_stream().wait_stream(side)
    sp.sp24_adamw(a, g, sa, 1, grad_scale=scale, seed=4, **{**HYPER, "lr": lr.item()})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        sp.sp24_adamw(b, g, sb, step, grad_scale=scale, seed=4, **hyper)
    for k in range(2, 5):
        for i, x in enumerate(g):
            x.copy_(rand(10 * k + i, x.numel()))
        lr.fill_(1e-2 / k), scale.fill_(0.1 * k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert step.item() == k
        sp.sp24_adamw(a, g, sa, k, grad_scale=scale, seed=4, **{**HYPER, "lr": lr.item()})
        for x, y in zip(a, b):  # bias corrections of the device's own pow: a unit in the last place of the rate
            assert ((x - y).abs() <= 4 * ref.U * (x.abs() + 1)).all()
        for s, t in zip(sa, sb):
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(s, t))


def test_grad_scale_and_betas():
    say("adamw scale and betas")
    for bits in (32, 8):
        for betas, scale in (((0.0, 0.0), 3.0), ((0.95, 0.9), 0.125), ((0.5, 0.999999), 1e-3)):
            p, g = rand(1, 3000), rand(2, 3000, dtype=torch.bfloat16)
            state = sp.sp24_adamw_state(p, bits)
            hyper = {**HYPER, "betas": betas}
            for step in (1, 2, 1000):
                want = expect(p, g, state, step, seed=5, scale=scale, **hyper)
                sp.sp24_adamw([p], [g], [state], step, grad_scale=torch.tensor(scale, device="cuda"), seed=5, **hyper)
                check(p, state, *want)


def test_large_tensor_and_offsets():
    """Elements past 2^31 bytes and the last chunk of a large tensor."""
    say("adamw 600 million elements")
    n = 600_000_003
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[:4096], g[-4099:] = rand(1, 4096), rand(2, 4099)
    state = sp.sp24_adamw_state(p, 8)
    sp.sp24_adamw([p], [g], [state], 1, seed=6, **HYPER)
    r = ref.random_words(6, 1, 0, n)[-4099:]
    m, v = ref.moments(np.zeros(4099, np.float32), np.zeros(4099, np.float32), host(g[-4099:]), 0.9, 0.999)
    lead = (n - 4099) % 128  # elements of the first block before the tail
    pad = lambda x: np.concatenate([np.zeros(lead, x.dtype), x])  # noqa: E731
    mc, ms = ref.first_codes(pad(m), pad(r & 0xFFFF))
    vc, vs = ref.second_codes(pad(v), pad(r >> 16))
    assert np.array_equal(host(state[0][-4099:]), mc[lead:]) and np.array_equal(host(state[2][-4099:]), vc[lead:])
    assert np.array_equal(host(state[1][-len(ms):]), ms) and np.array_equal(host(state[3][-len(vs):]), vs)
    assert (p[4096:-4099] == 0).all() and (p[:4096] != 0).all() and (p[-4099:] != 0).all()


def test_refusals():
    say("adamw refuses")
    p, g = rand(1, 64), rand(2, 64)
    s32, s8 = sp.sp24_adamw_state(p), sp.sp24_adamw_state(p, 8)
    ok = dict(params=[p], grads=[g], states=[s32], step=1)
    for bad in (dict(grads=[]), dict(params=[p.half()]), dict(grads=[g.double()]), dict(grads=[g[:32]]), dict(grads=[g.cpu()]),
                dict(states=[s32[:1]]), dict(states=[(s32[0], s32[1].half())]), dict(states=[s8[:3]]), dict(params=[rand(3, 128)[::2]]),
                dict(copies=[g]), dict(copies=[g.half()[:3]]), dict(params=[p, p], grads=[g, g], states=[s32, s32]),
                dict(params=[p, rand(4, 64)], grads=[g, g.half()], states=[s32, sp.sp24_adamw_state(p)]),
                dict(params=[p, rand(4, 64)], grads=[g, g], states=[s32, s8]), dict(step=torch.ones(1, device="cuda")),
                dict(lr=torch.ones(1, dtype=torch.float64, device="cuda")), dict(grad_scale=torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            sp.sp24_adamw(**{**ok, **bad})
    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=0.0), dict(weight_decay=-1.0),
                dict(params=[rand(5, 65)[1:]])):
        with pytest.raises(sp.Sp24Error):
            sp.sp24_adamw(**{**ok, **bad})
    with pytest.raises(TypeError):
        sp.sp24_adamw(**{**ok, "grad_scale": 2.0})
    with pytest.raises(ValueError):
        sp.sp24_adamw_state(p, 16)
    sp.sp24_adamw([], [], [], 1)
    sp.sp24_adamw([p], [None], [s32], 1)
