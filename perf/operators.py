"""Measured cases of the 8-bit operators around a 2:4-sparse Linear layer.

Activations and weights are held as 8-bit floating-point codes (e4m3) with one power-of-two scale (e8m0)
for each block of 128: 128 consecutive channels of a token, or 128 x 128 of a weight. The operators:

  norm       h = x + r;  y = h / sqrt(mean(h^2) + eps) * gamma;  y as codes and scales
  norm_back  the gradients of x (and r) and of gamma, from that of y and that of h
  quant      x as codes and scales: the layer's input when no norm precedes it, and the copy of an
             activation that is kept for the backward pass
  gemm       Y = X W^T with W 2:4 sparse, both operands as codes and scales
  wgrad      dW = dY^T X from the kept 8-bit X, at all weights or only at those that the 2:4 pattern keeps

With `own` false, run() computes them from elementary torch operations in 32 bits; with `own` true it calls
the library.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token between two layers: nothing but latency
        {"name": "norm, one token", "op": "norm", "n": 1, "k": 4096, "type": "bf16", "residual": True},
        # an image encoder's batch: 32 images of 197 tokens, short rows, no residual to add
        {"name": "norm, short rows", "op": "norm", "n": 6304, "k": 768, "type": "bf16", "residual": False},
        # a training batch or a long prompt at the widest layer input
        {"name": "norm, wide rows", "op": "norm", "n": 8192, "k": 8192, "type": "bf16", "residual": True},
        # fine-tuning on single images, master precision
        {"name": "norm_back, few rows", "op": "norm_back", "n": 197, "k": 768, "type": "fp32", "residual": True},
        {"name": "norm_back, wide rows", "op": "norm_back", "n": 8192, "k": 8192, "type": "bf16", "residual": True},
        # the input of a down projection: few sequences decoding, and a whole training batch
        {"name": "quant, 16 tokens", "op": "quant", "n": 16, "k": 11008, "type": "bf16"},
        {"name": "quant, batch", "op": "quant", "n": 8191, "k": 11008, "type": "fp16"},
        # decoding one sequence; decoding a ragged batch with the widest weight; a training step's product
        {"name": "gemm, one token", "op": "gemm", "m": 4096, "k": 4096, "n": 1, "out": "bf16"},
        {"name": "gemm, 37 tokens", "op": "gemm", "m": 11008, "k": 4096, "n": 37, "out": "fp16"},
        {"name": "gemm, batch", "op": "gemm", "m": 28672, "k": 8192, "n": 8192, "out": "bf16"},
        # a small layer with many tokens: few outputs, a long sum; a projection with its pattern kept
        {"name": "wgrad, small layer", "op": "wgrad", "m": 768, "k": 768, "n": 6304, "out": "fp32", "masked": False},
        {"name": "wgrad, projection", "op": "wgrad", "m": 11008, "k": 4096, "n": 4096, "out": "bf16", "masked": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _k(rng, lo, hi):
    """Channels: a multiple of 16, of 128 half of the time."""
    step = rng.choice([16, 128])
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_back", "quant", "gemm", "gemm", "wgrad"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_back", "quant"):
        k = _k(rng, 256, 16384)
        c = {"op": op, "n": _log(rng, 1, 8192 * 4096 // k), "k": k, "type": kind}
        if op != "quant":
            c["residual"] = rng.random() < 0.7
        return c
    if op == "gemm":
        # up to the listed weights; single tokens, small batches and whole prompts alike
        m, k = _log(rng, 512, 28672), _k(rng, 512, 8192)
        n = rng.choice([_log(rng, 1, 16), _log(rng, 17, 300), _log(rng, 300, 6304)])
        return {"op": op, "m": m, "k": k, "n": n, "out": rng.choice(["bf16", "fp16"])}
    m, k = _log(rng, 512, 11008) // 8 * 8, _k(rng, 512, 8192)
    return {"op": op, "m": m, "k": k, "n": _log(rng, 1, 6304), "out": rng.choice(["bf16", "fp32"]),
            "masked": rng.random() < 0.5}


def work(case):
    """Each input read once, each output written once; products of kept weights only."""
    op, n, k = case["op"], case["n"], case["k"]
    kb = -(-k // BLOCK)
    if op in ("norm", "norm_back", "quant"):
        e = TYPES[case["type"]].itemsize
        codes = n * k + n * kb
        if op == "quant":
            return {"bytes": n * k * e + codes, "flops": 2 * n * k}
        res = case["residual"]
        if op == "norm":  # x, r, gamma in; codes, scales, h, rstd out
            return {"bytes": n * k * e * (3 if res else 1) + k * e + codes + 4 * n, "flops": 5 * n * k}
        # dy, h, dh, gamma, rstd in; dx, dgamma out
        return {"bytes": n * k * e * (4 if res else 3) + k * e + 4 * n + 4 * k, "flops": 10 * n * k}
    m, o = case["m"], TYPES[case["out"]].itemsize
    if op == "gemm":
        weight = m * k // 2 + m * k // 8 + -(-m // BLOCK) * kb
        return {"bytes": weight + n * k + n * kb + n * m * o, "flops": m * n * k}
    return {"bytes": 2 * n * m + n * k + n * kb + m * k * o + (m * k // 8 if case["masked"] else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------------------ inputs


def _codes(y):
    """y (n x k, fp32) as e4m3 codes and e8m0 scales of each 128 channels, the scale the least power of two
    that keeps the block's largest magnitude within 448."""
    n, k = y.shape
    kb = -(-k // BLOCK)
    blocks = (torch.nn.functional.pad(y, (0, -k % BLOCK)) if k % BLOCK else y).view(n, kb, BLOCK)
    big = blocks.abs().amax(2)
    # 448 = 1.75 * 2^8: the exponent field less 8, one more where the fraction passes 0.75
    e = (((big.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=0)
    codes = (blocks * ((254 - e) << 23).view(torch.float32).unsqueeze(2)).view(n, -1)[:, :k].to(torch.float8_e4m3fn)
    return codes, torch.where(big.isfinite(), e, 255).to(torch.uint8).view(torch.float8_e8m0fnu)


def _kept(w):
    """Which two of each four consecutive weights have the largest magnitudes; lower index wins ties."""
    m, k = w.shape
    a = w.abs().view(m, k // 4, 4).unbind(2)
    ranks = []
    for t in range(4):
        beaten = sum((a[u] >= a[t]).int() if u < t else (a[u] > a[t]).int() for u in range(4) if u != t)
        ranks.append(beaten < 2)
    return torch.stack(ranks, 2)  # m x k/4 x 4


def _positions(kept):
    """The two kept positions of each group (int64), ascending."""
    first = kept.int().argmax(2)
    last = 3 - kept.flip(2).int().argmax(2)
    return first, last


def _tiles(rows, unit):
    """Row-major bytes (m x b, m a multiple of 16, b of 4 `unit`) in the library's tiled order: 16 rows x 4 unit
    bytes, stored quarter by quarter."""
    m, b = rows.shape
    return rows.view(m // 16, 16, b // (4 * unit), 4, unit).permute(0, 2, 3, 1, 4).contiguous().view(-1)


def _meta(kept):
    m, g = kept.shape[:2]
    first, last = _positions(kept)
    nib = (first | (last << 2)).to(torch.uint8)
    nib = torch.nn.functional.pad(nib, (0, -g % 32, 0, -m % 16), value=4)
    return _tiles(nib[:, 0::2] | (nib[:, 1::2] << 4), 4)


def _values(codes, kept):
    m, k = codes.shape
    byte = codes.view(torch.uint8).view(m, k // 4, 4)
    first, last = _positions(kept)
    v = torch.stack([byte.gather(2, first.unsqueeze(2)).squeeze(2), byte.gather(2, last.unsqueeze(2)).squeeze(2)], 2).view(m, k // 2)
    v = torch.nn.functional.pad(v, (0, -k % 128 // 2, 0, -m % 16))
    return _tiles(v, 16).view(torch.float8_e4m3fn)


def _weight(m, k, g):
    """A trained weight's spread, pruned and coded with one scale for each 128 x 128."""
    w = torch.randn(m, k, generator=g, device="cuda").mul_(0.02)
    kept = _kept(w)
    w = w.mul_(kept.view(m, k))
    big = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -m % BLOCK))
    big = big.view(big.shape[0] // BLOCK, BLOCK, big.shape[1] // BLOCK, BLOCK).abs().amax((1, 3))
    f, p = torch.frexp(big)
    e = torch.where(f > 0.875, p - 8, p - 9)
    w = w * torch.ldexp(torch.ones((), device="cuda"), -e).repeat_interleave(BLOCK, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return w.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), kept


def _activations(n, k, g, dtype=torch.float32):
    """Channels of unequal size, as in a transformer's residual stream."""
    return (torch.randn(n, k, generator=g, device="cuda") * torch.randn(k, generator=g, device="cuda").mul_(0.5).exp_()).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, n, k = case["op"], case["n"], case["k"]
    s = {"case": case}
    if op in ("norm", "norm_back", "quant"):
        dt = TYPES[case["type"]]
        s["x"] = _activations(n, k, g, dt)
        if op == "quant":
            return s
        s["gamma"] = (1 + 0.1 * torch.randn(k, generator=g, device="cuda")).to(dt)
        if op == "norm":
            s["r"] = _activations(n, k, g, dt) if case["residual"] else None
        else:
            s["rstd"] = s["x"].float().square().mean(1).add(EPS).rsqrt()
            s["dy"] = torch.randn(n, k, generator=g, device="cuda").to(dt)
            s["dh"] = torch.randn(n, k, generator=g, device="cuda").to(dt) if case["residual"] else None
        return s
    s["x"], s["xs"] = _codes(_activations(n, k, g))
    m = case["m"]
    if op == "gemm":
        s["w"], s["ws"], kept = _weight(m, k, g)
        s["values"], s["meta"] = _values(s["w"], kept), _meta(kept)
        return s
    s["dy"] = torch.randn(n, m, generator=g, device="cuda").to(torch.bfloat16)
    s["kept"] = s["meta"] = None
    if case["masked"]:
        kept = _kept(torch.randn(m, k, generator=g, device="cuda"))
        s["kept"], s["meta"] = kept.view(m, k), _meta(kept)
    return s


# ------------------------------------------------------------------------------------------ one pass


def _plain_norm(s):
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    hf = h.float()
    rstd = (hf.square().mean(1) + EPS).rsqrt()
    codes, scales = _codes(hf * rstd.unsqueeze(1) * s["gamma"].float())
    return {"codes": codes, "scales": scales, "h": None if s["r"] is None else h, "rstd": rstd}


def _plain_norm_back(s):
    rstd = s["rstd"].unsqueeze(1)
    xhat, dy = s["x"].float() * rstd, s["dy"].float()
    gdy = dy * s["gamma"].float()
    dx = rstd * (gdy - xhat * (gdy * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0)}


def _values_of(codes, scales):
    """Codes (n x k) with a scale for each 128 channels, as fp32."""
    return codes.float() * scales.float().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _plain_gemm(s):
    m, k = s["w"].shape
    w = s["w"].float() * s["ws"].float().repeat_interleave(BLOCK, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return (_values_of(s["x"], s["xs"]) @ w.t()).to(TYPES[s["case"]["out"]])


def _plain_wgrad(s):
    dw = s["dy"].float().t() @ _values_of(s["x"], s["xs"])
    if s["kept"] is not None:
        dw = dw * s["kept"]
    return dw.to(TYPES[s["case"]["out"]])


def _plain_quant(s):
    codes, scales = _codes(s["x"].float())
    return {"codes": codes, "scales": scales}


def _own(s):
    import structured_sparse_gemm_sp24_amd as sp

    op = s["case"]["op"]
    if op == "norm":
        codes, scales, h, rstd = sp.sp24_rmsnorm_fp8(s["x"], s["gamma"], EPS, residual=s["r"])
        return {"codes": codes, "scales": scales, "h": None if s["r"] is None else h, "rstd": rstd}
    if op == "norm_back":
        dx, dgamma = sp.sp24_rmsnorm_backward(s["dy"], s["x"], s["rstd"], s["gamma"], dH=s["dh"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "quant":
        codes, scales = sp.sp24_quant_fp8(s["x"])
        return {"codes": codes, "scales": scales}
    out = TYPES[s["case"]["out"]]
    if op == "gemm":
        return {"y": sp.sp24_gemm_fp8(s["values"], s["meta"], s["ws"], s["case"]["m"], s["x"], s["xs"], out_dtype=out)}
    return {"dw": sp.sp24_grad_weight_fp8(s["dy"], s["x"], s["xs"], meta=s["meta"], out_dtype=out)}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_back":
        return _plain_norm_back(state)
    if op == "quant":
        return _plain_quant(state)
    if op == "gemm":
        return {"y": _plain_gemm(state)}
    return {"dw": _plain_wgrad(state)}


# ------------------------------------------------------------------------------------------ 64 bits


def _exact_codes(y):
    """Codes as the numbers that they stand for before scaling, and scales, from y in 64 bits."""
    n, k = y.shape
    codes, scales = torch.empty_like(y), torch.empty(n, -(-k // BLOCK), dtype=torch.float64, device=y.device)
    for b in range(scales.shape[1]):
        part = y[:, b * BLOCK:(b + 1) * BLOCK]
        big = part.abs().max(1).values
        # the least e with big <= 448 * 2^e
        e = torch.ceil(torch.log2(big.clamp(min=1e-300) / 448))
        e = torch.where(448 * torch.exp2(e - 1) >= big, e - 1, e)
        e = torch.where(448 * torch.exp2(e) < big, e + 1, e).clamp(min=-127)
        v = part / torch.exp2(e).unsqueeze(1)
        # e4m3: 3 bits after the leading one, the least normal number 2^-6
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(v / step) * step
        scales[:, b] = torch.exp2(e)
    return codes, scales


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        codes, scales = _exact_codes(s["x"].double())
        return {"codes": codes, "scales": scales}
    if op == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(s["x"].dtype).double()
        var = torch.linalg.vector_norm(h, dim=1) ** 2 / case["k"]
        rstd = 1 / torch.sqrt(var + EPS)
        codes, scales = _exact_codes(s["gamma"].double() * h * rstd[:, None])
        return {"codes": codes, "scales": scales, "h": None if s["r"] is None else h, "rstd": rstd}
    if op == "norm_back":
        h, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double()
        gd = s["gamma"].double() * dy
        inner = torch.linalg.vecdot(gd, h) * r ** 3 / case["k"]
        dx = gd * r[:, None] - h * inner[:, None]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dgamma": torch.mv((dy * h).t(), r)}

    def wide(scales, rows, cols):
        e = scales.view(torch.uint8).double() - 127
        i = torch.arange(rows, device="cuda") // (BLOCK if e.shape[0] != rows else 1)
        return torch.exp2(e)[i][:, torch.arange(cols, device="cuda") // BLOCK]

    n, m, k = case["n"], case["m"], case["k"]
    x = s["x"].double() * wide(s["xs"], n, k)
    if op == "gemm":
        return {"y": torch.matmul(x, (s["w"].double() * wide(s["ws"], m, k)).t())}
    dw = torch.matmul(s["dy"].double().t(), x)
    if s["kept"] is not None:
        dw[~s["kept"]] = 0
    return {"dw": dw}
