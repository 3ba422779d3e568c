"""Plain forms of the layer operators (include/sp24_layer.h), written from their definitions: activations and their slopes in
64 bits, and the AdamW step in numpy, its moments in fp32 with one rounding a step as the contract of the 8-bit states has them."""
import numpy as np
import torch

U = 2.0 ** -24
UNIT = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
ACTIVATIONS = ["none", "gelu", "relu", "silu"]


def act(z: torch.Tensor, name: str) -> torch.Tensor:
    """In 64 bits, with the limits at the infinities."""
    if name == "relu":
        return torch.where(z < 0, 0.0, z)
    if name == "gelu":
        return torch.where(z == -torch.inf, 0.0, torch.special.ndtr(z) * z)
    if name == "silu":
        return torch.where(z == -torch.inf, 0.0, torch.special.expit(z) * z)
    return z


def slope(z: torch.Tensor, name: str) -> torch.Tensor:
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        y = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    else:
        s = torch.special.expit(z)
        y = s + z * s * (1 - s)
    return torch.where(z == torch.inf, 1.0, torch.where(z == -torch.inf, 0.0, y))


def act_error(z: torch.Tensor, name: str) -> torch.Tensor:
    """Most that the fp32 activation of an fp32 z may be off. SiLU: the argument's product and constant 2 |z| U, exponential,
    sum, reciprocal (one unit each in the last place, 2 U) and product, 6 U; 1e-35 where e^-z or its reciprocal leave fp32."""
    if name == "gelu":
        off = 8 * U * z.abs()
    elif name == "silu":
        off = (6 + 3 * z.abs()) * U * act(z, "silu").abs() + 1e-35
    else:
        return torch.zeros_like(z)
    return torch.where(torch.isinf(z), 0.0, off)  # the limits are exact (infinity times zero has no bound)


def slope_error(z: torch.Tensor, name: str) -> torch.Tensor:
    """The same of the slope. GELU: erfc / 2 within 8 U, as the activation; z phi(z), at most 0.25: |z| <= 20 rounded in three
    products (3 U) and the exponential's argument (z^2 / 2 twice rounded: z^2 U, z^2 |z| phi below 0.47) and two units, 4 U
    in all; the sum 2 U. SiLU: s within (3 |z| + 5) U of itself; 1 - s off by that of s and U; z s (1 - s), at most 0.23, by
    (6 |z| + 14) U of itself in s and 1 - s, and |z| s (1 - s) |z| below 0.5; the sum 2 U: below 16 U in all."""
    return torch.full_like(z, {"gelu": 16 * U, "silu": 16 * U}.get(name, 0.0))


# ---------------------------------------------------------------- AdamW

def mix(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.uint32)
    with np.errstate(over="ignore"):
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x9E3779B9)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x6A09E667)
    return x ^ (x >> np.uint32(16))


def random_words(seed: int, step: int, index: int, n: int) -> np.ndarray:
    low = lambda v: np.uint32(v & 0xFFFFFFFF)  # noqa: E731
    key = mix(mix(mix(low(seed)) ^ low(seed >> 32)) ^ low(step))
    with np.errstate(over="ignore"):
        key = mix(key + low(index * 0x9E3779B9))
        return mix(np.arange(n, dtype=np.uint32) * np.uint32(0xBB67AE85) + key)


def per_block(x: np.ndarray) -> np.ndarray:
    x = x.reshape(-1)
    return np.pad(x, (0, -x.size % 128)).reshape(-1, 128)


def spread(s: np.ndarray, n: int) -> np.ndarray:
    return np.repeat(s, 128)[:n]


E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def first_codes(m: np.ndarray, r16: np.ndarray):
    """(codes as bytes, scale bytes) of finite fp32 m: with x = |m| / unit between the numbers lo and hi of the format, hi where
    r16 + (x - lo) / (hi - lo) 2^16 passes 2^16."""
    amax = np.abs(per_block(m)).max(1).astype(np.float64)
    e = np.ceil(np.log2(np.maximum(amax, 1e-300) / 448))
    e = np.where(448 * 2.0 ** (e - 1) >= amax, e - 1, e)
    e = np.maximum(np.where(448 * 2.0 ** e < amax, e + 1, e), -127)
    x = np.abs(m.astype(np.float64)) * 2.0 ** -spread(e, m.size)
    lo = np.searchsorted(E4M3, x, side="right") - 1
    step = np.append(np.diff(E4M3), 32.0)[lo]
    # the 20 cut bits of fp32 (below 2^-6: 20 bits below 2^-9, what is lower left out)
    part = np.floor((x - E4M3[lo]) / step * 2.0 ** 20)
    code = lo + (part + r16.astype(np.float64) * 16 >= 2.0 ** 20)
    return (code.astype(np.uint8) | np.where(np.signbit(m), 0x80, 0).astype(np.uint8)), (e + 127).astype(np.uint8)


def second_codes(v: np.ndarray, r16: np.ndarray):
    """(codes, scale bytes) of finite v >= 0: sqrt(v) / unit down, or up where r16 (2 c + 1) < (x - c^2) 2^16 in fp32."""
    f = np.float32
    vmax = per_block(v).max(1).astype(np.float64)
    e = np.full(vmax.shape, -63.0)
    while (bad := 65025.0 * 4.0 ** e < vmax).any():
        e = e + bad
    x = (v.astype(np.float64) * 4.0 ** -spread(e, v.size)).astype(f)
    c = np.floor(np.sqrt(x.astype(np.float64))).astype(f)
    up = r16.astype(f) * (f(2) * c + f(1)) < (x - c * c) * f(65536)
    return np.maximum(c + up, (v > 0).astype(f)).astype(np.uint8), (e + 127).astype(np.uint8)


def first_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    number = torch.from_numpy(codes.reshape(-1).copy()).view(torch.float8_e4m3fn).float().numpy()
    return (number.astype(np.float64) * 2.0 ** (spread(scales.astype(np.float64), codes.size) - 127)).astype(np.float32)


def second_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    e = np.maximum(spread(scales.astype(np.float64), codes.size) - 127, -63)
    return (codes.reshape(-1).astype(np.float64) ** 2 * 4.0 ** e).astype(np.float32)


def moments(m, v, g, b1, b2, scale=1.0):
    """New moments in fp32, one rounding a step."""
    f = np.float32
    g = (g.astype(f) * f(scale)).astype(f)
    return m * f(b1) + g * f(1 - b1), v * f(b2) + (g * g) * f(1 - b2)


def weights(p, m, v, step, lr, b1, b2, eps, decay):
    """New weights in 64 bits from the new moments."""
    m, v, p = (np.asarray(x, np.float64) for x in (m, v, p))
    return p * (1 - lr * decay) - lr / (1 - b1 ** step) * m / (np.sqrt(v) / np.sqrt(1 - b2 ** step) + eps)
