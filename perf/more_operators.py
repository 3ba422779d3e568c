"""Measured cases of the operators that finish a 2:4-sparse Linear layer and train it.

  linear       Y = act(W X + bias) + residual for a 2:4 weight in bf16, optionally with W X + bias for the backward pass
  linear_fp8   the same with weight and activations as 8-bit codes (e4m3) and power-of-two scales of blocks of 128
  back         the epilogue's gradient: dZ = dY act'(Z), and the bias's, its sum over tokens
  adamw        a step of AdamW over a list of tensors, states in 32 bits or in 8

8-bit states hold, for each 128 consecutive elements, the first moment as e4m3 codes and the root of the second as whole
numbers up to 255, both with a power-of-two scale; they are rounded up or down by 16 random bits, a hash of the step's seed,
the step, the tensor and the element.

With `own` false, run() computes them from elementary torch operations in 32 bits; with `own` true it calls the library.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.1


def listed():
    return [
        # decoding one sequence: a gate's projection
        {"name": "linear, one token", "op": "linear", "m": 11008, "k": 4096, "n": 1, "batch": 1, "layout": "token", "out": "bf16",
         "act": "silu", "residual": False, "pre": False},
        # an image encoder's attention output: 32 images of 197 tokens, back into the residual stream
        {"name": "linear, image tokens", "op": "linear", "m": 768, "k": 768, "n": 6304, "batch": 1, "layout": "token", "out": "bf16",
         "act": "none", "residual": True, "pre": False},
        # a training step's up projection, its pre-activation kept
        {"name": "linear, training", "op": "linear", "m": 11008, "k": 4096, "n": 4096, "batch": 1, "layout": "token", "out": "bf16",
         "act": "gelu", "residual": False, "pre": True},
        # 1 x 1 convolution that widens 28 x 28 images, added to the shortcut
        {"name": "linear, images", "op": "linear", "m": 512, "k": 128, "n": 784, "batch": 32, "layout": "feature", "out": "bf16",
         "act": "relu", "residual": True, "pre": False},
        # 16 sequences decoding: a down projection into the residual stream
        {"name": "linear_fp8, 16 tokens", "op": "linear_fp8", "m": 4096, "k": 11008, "n": 16, "out": "fp16",
         "act": "none", "residual": True, "pre": False},
        # a whole prompt or batch through the widest weight
        {"name": "linear_fp8, batch", "op": "linear_fp8", "m": 28672, "k": 8192, "n": 8192, "out": "bf16",
         "act": "gelu", "residual": False, "pre": False},
        # a ragged training batch, everything at once
        {"name": "linear_fp8, ragged", "op": "linear_fp8", "m": 11007, "k": 4096, "n": 1500, "out": "bf16",
         "act": "silu", "residual": True, "pre": True},
        # fine-tuning on single images in master precision
        {"name": "back, few rows", "op": "back", "n": 197, "m": 768, "type": "fp32", "act": "gelu"},
        {"name": "back, batch", "op": "back", "n": 8192, "m": 28672, "type": "bf16", "act": "silu"},
        # the first step of a small encoder block's vectors: many tensors, nothing but latency
        {"name": "adamw, vectors", "op": "adamw", "tensors": "+".join(["768"] * 12 + ["2304"] * 4), "bits": 32, "grad": "fp32",
         "copy": "", "step": 1},
        # a block's weights and vectors with 16-bit gradients and working copies
        {"name": "adamw, block", "op": "adamw", "tensors": "11008x4096+4096+11008x4096+4096x11008+11008+4096", "bits": 32, "grad": "bf16",
         "copy": "bf16", "step": 1000},
        # the widest block, its states in 8 bits
        {"name": "adamw, 8 bits", "op": "adamw", "tensors": "28672x8192+8192+8192x28672+28672", "bits": 8, "grad": "bf16",
         "copy": "bf16", "step": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _k(rng, lo, hi, steps):
    step = rng.choice(steps)
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_fp8", "linear_fp8", "back", "adamw", "adamw"])
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if op in ("linear", "linear_fp8"):
        c = {"op": op, "act": act, "residual": rng.random() < 0.5, "pre": act != "none" and rng.random() < 0.4}
        if op == "linear" and rng.random() < 0.25:
            # images of up to 56 x 56, each row on 16 bytes
            n = _log(rng, 8, 392) * 8
            return {**c, "m": _log(rng, 64, 2048), "k": _k(rng, 64, 2048, [16, 64]), "n": n, "batch": _log(rng, 1, max(2, 25088 // n)),
                    "layout": "feature", "out": rng.choice(["bf16", "fp32"])}
        c["m"], c["n"] = _log(rng, 512, 28672), rng.choice([_log(rng, 1, 16), _log(rng, 17, 300), _log(rng, 300, 6304)])
        if rng.random() < 0.5:
            c["m"] = c["m"] // 16 * 16
        if op == "linear":
            return {**c, "k": _k(rng, 512, 8192, [64, 128]), "batch": 1, "layout": "token", "out": rng.choice(["bf16", "bf16", "fp32"])}
        return {**c, "k": _k(rng, 512, 8192, [16, 128]), "out": rng.choice(["bf16", "fp16"])}
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "back":
        m = _log(rng, 256, 28672)
        return {"op": op, "n": _log(rng, 1, 8192 * 8192 // m), "m": m, "type": kind, "act": act}
    shapes = []
    for _ in range(rng.randint(1, 8)):
        m, k = _log(rng, 1, 4096), _log(rng, 16, 8192)
        shapes.append(rng.choice(["%dx%d" % (m, k), "%d" % m]))
    return {"op": op, "tensors": "+".join(shapes), "bits": rng.choice([8, 32]), "grad": kind, "copy": rng.choice(["", "bf16", "fp16"]),
            "step": rng.choice([1, 7, 300, 20000])}


def _shapes(case):
    return [[int(d) for d in t.split("x")] for t in case["tensors"].split("+")]


def work(case):
    """Each input read once, each output written once; products of kept weights only."""
    op = case["op"]
    if op == "back":
        n, m, e = case["n"], case["m"], TYPES[case["type"]].itemsize
        if case["act"] == "none":  # the bias's gradient alone
            return {"bytes": n * m * e + 4 * m, "flops": n * m}
        return {"bytes": 3 * n * m * e + 4 * m, "flops": 10 * n * m}
    if op == "adamw":
        total = sum(math.prod(s) for s in _shapes(case))
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        each = 8 + TYPES[case["grad"]].itemsize + state + (TYPES[case["copy"]].itemsize if case["copy"] else 0)
        return {"bytes": int(total * each), "flops": 15 * total}
    m, k, n, o = case["m"], case["k"], case["n"], TYPES[case["out"]].itemsize
    outs = 1 + case["residual"] + case["pre"]
    if op == "linear":
        n *= case["batch"]
        return {"bytes": m * k + m * k // 8 + 2 * n * k + 4 * m + outs * n * m * o, "flops": m * n * k}
    kb = -(-k // BLOCK)
    weight = m * k // 2 + m * k // 8 + -(-m // BLOCK) * kb
    return {"bytes": weight + n * k + n * kb + 4 * m + outs * n * m * o, "flops": m * n * k}


# ------------------------------------------------------------------------------------------ inputs


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(n, k, g):
    """Channels of unequal size, as in a transformer's residual stream."""
    return _rand(g, n, k) * _rand(g, k).mul_(0.5).exp_()


def _kept(w):
    """Which two of each four consecutive weights have the largest magnitudes; lower index wins ties."""
    m, k = w.shape
    a = w.abs().view(m, k // 4, 4).unbind(2)
    ranks = []
    for t in range(4):
        beaten = sum((a[u] >= a[t]).int() if u < t else (a[u] > a[t]).int() for u in range(4) if u != t)
        ranks.append(beaten < 2)
    return torch.stack(ranks, 2)  # m x k/4 x 4


def _tiles(rows, unit):
    """Row-major bytes (m x b, m a multiple of 16, b of 4 `unit`) in the library's tiled order: 16 rows x 4 unit
    bytes, stored quarter by quarter."""
    m, b = rows.shape
    return rows.view(m // 16, 16, b // (4 * unit), 4, unit).permute(0, 2, 3, 1, 4).contiguous().view(-1)


def _compressed(w, kept):
    """(values, metadata) of a pruned weight of one or two bytes a value, in the library's order."""
    m, k = w.shape
    e = w.element_size()
    tile = 128 // e  # dense columns a tile
    first = kept.int().argmax(2)
    last = 3 - kept.flip(2).int().argmax(2)
    nib = (first | (last << 2)).to(torch.uint8)
    nib = torch.nn.functional.pad(nib, (0, -k % tile // 4, 0, -m % 16), value=4)
    raw = w.view(torch.uint8 if e == 1 else torch.int16).view(m, k // 4, 4)
    v = torch.stack([raw.gather(2, first.unsqueeze(2)).squeeze(2), raw.gather(2, last.unsqueeze(2)).squeeze(2)], 2).view(m, k // 2)
    v = torch.nn.functional.pad(v, (0, -k % tile // 2, 0, -m % 16)).view(torch.uint8)
    return _tiles(v, 16).view(w.dtype), _tiles(nib[:, 0::2] | (nib[:, 1::2] << 4), tile // 32)


def _codes(y):
    """y (n x k, fp32) as e4m3 codes and e8m0 scales of each 128 channels, the scale the least power of two
    that keeps the block's largest magnitude within 448."""
    n, k = y.shape
    kb = -(-k // BLOCK)
    blocks = (torch.nn.functional.pad(y, (0, -k % BLOCK)) if k % BLOCK else y).view(n, kb, BLOCK)
    e = _code_scale(blocks.abs().amax(2))
    codes = (blocks * ((254 - e) << 23).view(torch.float32).unsqueeze(2)).view(n, -1)[:, :k].to(torch.float8_e4m3fn)
    return codes, e.to(torch.uint8).view(torch.float8_e8m0fnu)


def _code_scale(big):
    # 448 = 1.75 * 2^8: the exponent field less 8, one more where the fraction passes 0.75
    return (((big.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=0)


def _weight_fp8(w):
    """A pruned weight as e4m3 codes with one scale for each 128 x 128."""
    m, k = w.shape
    big = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -m % BLOCK))
    big = big.view(big.shape[0] // BLOCK, BLOCK, big.shape[1] // BLOCK, BLOCK).abs().amax((1, 3))
    e = _code_scale(big)
    unit = ((254 - e) << 23).view(torch.float32)
    w = w * unit.repeat_interleave(BLOCK, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return w.to(torch.float8_e4m3fn), e.to(torch.uint8).view(torch.float8_e8m0fnu)


def _prepare_linear(case, g, s):
    m, k, n, out = case["m"], case["k"], case["n"], TYPES[case["out"]]
    w = _rand(g, m, k).mul_(0.02)
    kept = _kept(w)
    w = w.mul_(kept.view(m, k))
    s["bias"] = _rand(g, m).mul_(0.2)
    if case["op"] == "linear":
        s["w"] = w.to(torch.bfloat16)
        s["values"], s["meta"] = _compressed(s["w"], kept)
        x = _activations(n * case["batch"], k, g)
        if case["layout"] == "token":
            s["x"], y = x.to(torch.bfloat16), (n, m)
        else:
            s["x"], y = x.view(case["batch"], n, k).transpose(1, 2).to(torch.bfloat16, memory_format=torch.contiguous_format), (case["batch"], m, n)
    else:
        s["w"], s["ws"] = _weight_fp8(w)
        s["values"], s["meta"] = _compressed(s["w"], kept)
        s["x"], s["xs"] = _codes(_activations(n, k, g))
        y = (n, m)
    s["r"] = _rand(g, *y).to(out) if case["residual"] else None


def _prepare_adamw(case, g, s):
    """Weights, gradients whose sizes vary from element to element, and the moments that such gradients leave."""
    first = case["step"] == 1
    s["p"], s["g"], s["state"] = [], [], []
    for shape in _shapes(case):
        size = _rand(g, *shape).mul_(0.7).exp_().mul_(1e-3)
        s["p"].append(_rand(g, *shape).mul_(0.02))
        s["g"].append(_rand(g, *shape).mul_(size).to(TYPES[case["grad"]]))
        m = torch.zeros_like(size) if first else _rand(g, *shape).mul_(size).mul_(0.2)
        v = torch.zeros_like(size) if first else size.square_()
        if case["bits"] == 32:
            s["state"].append((m, v))
        else:
            half = torch.full((m.numel(),), 1 << 15, dtype=torch.int64, device="cuda")
            s["state"].append((*_first_codes(m, half), *_second_codes(v, half)))
    s["seed"] = int(torch.randint(1 << 60, (1,), generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "back":
        shape, dt = (case["n"], case["m"]), TYPES[case["type"]]
        s["dy"] = _rand(g, *shape).to(dt)
        s["z"] = None if case["act"] == "none" else _rand(g, *shape).mul_(2).to(dt)
    elif case["op"] == "adamw":
        _prepare_adamw(case, g, s)
    else:
        _prepare_linear(case, g, s)
    return s


# ------------------------------------------------------------------------------------------ one pass


def _act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z / (1 + torch.exp(-z)) if name == "silu" else z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).float()
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _plain_linear(s):
    c = s["case"]
    out, token = TYPES[c["out"]], c["op"] == "linear_fp8" or c["layout"] == "token"
    if c["op"] == "linear":
        w, x = s["w"].float(), s["x"].float()
    else:
        m, k = s["w"].shape
        w = s["w"].float() * s["ws"].float().repeat_interleave(BLOCK, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
        x = s["x"].float() * s["xs"].float().repeat_interleave(BLOCK, 1)[:, :k]
    z = x @ w.t() + s["bias"] if token else w @ x + s["bias"].unsqueeze(1)
    y = _act(z, c["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(out), "z": z.to(out) if c["pre"] else None}


def _plain_back(s):
    dy, act = s["dy"].float(), s["case"]["act"]
    if act == "none":
        return {"dz": None, "dbias": dy.sum(0)}
    dz = dy * _act_slope(s["z"].float(), act)
    return {"dz": dz.to(s["dy"].dtype), "dbias": dz.sum(0)}


def _low(x):
    return x & 0xFFFFFFFF


def _mix(x):
    """32 bits stirred; on whole numbers and on tensors of them alike (int64, kept within 32 bits)."""
    x = _low((x ^ (x >> 16)) * 0x9E3779B9)
    x = _low((x ^ (x >> 15)) * 0x6A09E667)
    return x ^ (x >> 16)


def _bits32(seed, step, tensor, n):
    """A random word for each element: 16 bits for each of the two moments."""
    key = _mix(_mix(_mix(_low(seed)) ^ (seed >> 32)) ^ _low(step))
    key = _mix(_low(key + tensor * 0x9E3779B9))
    i = torch.arange(n, dtype=torch.int64, device="cuda")
    return _mix(_low(_low(i) * 0xBB67AE85 + (i >> 32) * 0x9E3779B9 + key))


def _blocks(x):
    return torch.nn.functional.pad(x.reshape(-1), (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _spread(per_block, n):
    return per_block.repeat_interleave(BLOCK)[:n]


def _power(e):
    """2^e as fp32, for whole e from -126 to 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _first_codes(m, r16):
    """Codes (e4m3) and scales of the first moment: down to the next code, or up with the odds that keep it right on average."""
    n, flat = m.numel(), m.reshape(-1)
    e = _code_scale(_blocks(flat.abs()).amax(1))
    x = flat.abs() * ((254 - _spread(e, n)) << 23).view(torch.float32)
    r20 = (r16 << 4).to(torch.int32)
    code = torch.where(x < 2.0 ** -6, ((x * 2.0 ** 29).to(torch.int32) + r20) >> 20, ((x.view(torch.int32) + r20) >> 20) - 960)
    code = code.to(torch.uint8) | ((flat.view(torch.int32) >> 24) & 0x80).to(torch.uint8)
    return code.view(torch.float8_e4m3fn).view(m.shape), e.to(torch.uint8).view(torch.float8_e8m0fnu)


def _second_codes(v, r16):
    """Root of the second moment as whole numbers up to 255 of a power of two, at least 1 unless it is zero; up or down with
    the odds that keep the moment itself right on average."""
    n, flat = v.numel(), v.reshape(-1)
    # the least even k with max <= 255^2 2^k; 0x477E0100 is 255^2
    k = (_blocks(flat).amax(1).view(torch.int32) - 0x477E0100 + 0x7FFFFF) >> 23
    e = ((k + 1) >> 1).clamp(min=-63)
    x = flat * _power(-2 * _spread(e, n))
    c = torch.floor(torch.sqrt(x))
    up = r16.float() * (2 * c + 1) < (x - c * c) * 65536
    code = torch.maximum(c + up, (flat > 0).float())
    return code.to(torch.uint8).view(v.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _moments(state, n):
    if len(state) == 2:
        return state[0], state[1]
    mc, ms, vc, vs = state
    m = mc.float() * _spread(ms.float(), n).view(mc.shape)
    e = (vs.view(torch.uint8).int() - 127).clamp(min=-63)
    return m, vc.float() * vc.float() * _spread(_power(2 * e), n).view(vc.shape)


def _plain_adamw(s):
    c = s["case"]
    rate = LR / (1 - BETA1 ** c["step"])
    root = 1 / math.sqrt(1 - BETA2 ** c["step"])
    got = {"p": [], "state": [], "copy": []}
    for t, (p, g, state) in enumerate(zip(s["p"], s["g"], s["state"])):
        n, g = p.numel(), g.float()
        m, v = _moments(state, n)
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + (g * g) * (1 - BETA2)
        p = p * (1 - LR * DECAY) - rate * m / (torch.sqrt(v) * root + EPS)
        if c["bits"] == 8:
            r = _bits32(s["seed"], c["step"], t, n)
            got["state"].append((*_first_codes(m, r & 0xFFFF), *_second_codes(v, r >> 16)))
        else:
            got["state"].append((m, v))
        got["p"].append(p)
        got["copy"].append(p.to(TYPES[c["copy"]]) if c["copy"] else None)
    return got


def _own_adamw(sp, s):
    c = s["case"]
    p = [torch.empty_like(x) for x in s["p"]]
    state = [tuple(torch.empty_like(x) for x in t) for t in s["state"]]
    copies = [torch.empty_like(x, dtype=TYPES[c["copy"]]) for x in p] if c["copy"] else None
    sp.sp24_adamw(s["p"], s["g"], s["state"], step=c["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                  seed=s["seed"], copies=copies, out=(p, state))
    return {"p": p, "state": state, "copy": copies or [None] * len(p)}


def _own(s):
    import structured_sparse_gemm_sp24_amd as sp

    c = s["case"]
    if c["op"] == "adamw":
        return _own_adamw(sp, s)
    if c["op"] == "back":
        dz, dbias = sp.sp24_epilogue_backward(s["dy"], s["z"], activation=c["act"])
        return {"dz": None if c["act"] == "none" else dz, "dbias": dbias}
    how = {"bias": s["bias"], "activation": c["act"], "residual": s["r"], "preact": c["pre"], "out_dtype": TYPES[c["out"]]}
    if c["op"] == "linear":
        got = sp.sp24_gemm_bf16_fused(s["values"], s["meta"], c["m"], s["x"], layout=c["layout"], **how)
    else:
        got = sp.sp24_gemm_fp8_fused(s["values"], s["meta"], s["ws"], c["m"], s["x"], s["xs"], **how)
    return {"y": got[0], "z": got[1]} if c["pre"] else {"y": got, "z": None}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "adamw":
        return _plain_adamw(state)
    return _plain_back(state) if op == "back" else _plain_linear(state)


# ------------------------------------------------------------------------------------------ 64 bits


def _exact_linear(s):
    c = s["case"]
    m, k = s["w"].shape

    def wide(scales, rows):
        e = torch.exp2(scales.view(torch.uint8).double() - 127)
        i = torch.arange(rows, device="cuda") // (BLOCK if e.shape[0] != rows else 1)
        return e[i][:, torch.arange(k, device="cuda") // BLOCK]

    w, x = s["w"].double(), s["x"].double()
    if c["op"] == "linear_fp8":
        w, x = w * wide(s["ws"], m), x * wide(s["xs"], c["n"])
    if c["op"] == "linear_fp8" or c["layout"] == "token":
        z = torch.matmul(x, w.t()).add_(s["bias"].double())
    else:
        z = torch.stack([torch.matmul(w, one) for one in x]).add_(s["bias"].double()[:, None])
    if c["act"] == "relu":
        y = torch.where(z > 0, z, 0.0)
    elif c["act"] == "gelu":
        y = z * torch.special.ndtr(z)
    else:
        y = z * torch.special.expit(z) if c["act"] == "silu" else z
    return {"y": y if s["r"] is None else y + s["r"].double(), "z": z if c["pre"] else None}


def _exact_back(s):
    dy = s["dy"].double()
    act = s["case"]["act"]
    if act == "none":
        return {"dz": None, "dbias": torch.mv(dy.t(), torch.ones(dy.shape[0], dtype=torch.float64, device="cuda"))}
    z = s["z"].double()
    if act == "relu":
        slope = torch.sign(z).clamp(min=0)
    elif act == "gelu":
        slope = torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    else:
        half = torch.tanh(z / 2)
        slope = (1 + half) / 2 + z * (1 - half * half) / 4
    return {"dz": dy * slope, "dbias": torch.linalg.vecdot(dy.t(), slope.t())}


def _exact_first(m, word):
    """Codes as numbers before scaling, and scales."""
    flat = m.reshape(-1)
    pad = torch.zeros(-flat.numel() % BLOCK, dtype=torch.float64, device="cuda")
    big = torch.cat([flat.abs(), pad]).view(-1, BLOCK).max(1).values
    e = torch.ceil(torch.log2(big.clamp(min=1e-300) / 448))
    e = torch.where(448 * torch.exp2(e - 1) >= big, e - 1, e)
    e = torch.where(448 * torch.exp2(e) < big, e + 1, e).clamp(min=-127)
    x = flat.abs() * torch.exp2(-e)[torch.arange(flat.numel(), device="cuda") // BLOCK]
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    code = torch.floor(x / step + (word & 0xFFFF).double() / 65536) * step
    return (code * torch.sign(flat)).view(m.shape), torch.exp2(e)


def _exact_adamw(s):
    c = s["case"]
    t = c["step"]
    got = {"p": [], "state": [], "copy": []}
    for i, (p, g, state) in enumerate(zip(s["p"], s["g"], s["state"])):
        g, n = g.double(), p.numel()
        if c["bits"] == 32:
            m, v = state[0].double(), state[1].double()
        else:
            at = torch.arange(n, device="cuda") // BLOCK
            unit = [torch.exp2(x.view(torch.uint8).double() - 127)[at].view(p.shape) for x in (state[1], state[3])]
            m, v = state[0].double() * unit[0], (state[2].double() * unit[1]) ** 2
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g.square(), v, BETA2)
        move = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS) + DECAY * p.double()
        now = p.double() - LR * move
        got["p"].append(now)
        got["copy"].append(now if c["copy"] else None)
        got["state"].append((m, v) if c["bits"] == 32 else (*_exact_first(m, _bits32(s["seed"], t, i, n)), None, None))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    return _exact_back(s) if case["op"] == "back" else _exact_linear(s)
