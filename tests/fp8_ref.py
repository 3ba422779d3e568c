"""Plain 64-bit forms of the 8-bit floating-point operators (include/sp24_fp8.h), in numpy on the host, written from
their definitions, with error bounds of the fp32 kernels."""
import numpy as np
import torch

U32, U16, UB = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8  # unit roundoffs: fp32, fp16, bf16
UNIT = {torch.float32: U32, torch.float16: U16, torch.bfloat16: UB}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 number (ties to even) of magnitudes up to 448: 4 significant bits, least normal 2^-6."""
    a = np.maximum(np.abs(v), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(a)) - 3)
    return np.rint(v / step) * step


def scale_exp(amax: np.ndarray) -> np.ndarray:
    """The least e >= -127 with amax <= 448 * 2^e."""
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(np.maximum(amax, 1e-300) / 448)), -127)
    e = np.where(448 * 2.0 ** (e - 1) >= amax, e - 1, e)
    e = np.where(448 * 2.0 ** e < amax, e + 1, e)
    return np.maximum(e, -127)


def blocks(y: np.ndarray) -> np.ndarray:
    """N x K as N x ceil(K / 128) x 128, zeros after the row's end."""
    n, k = y.shape
    return np.pad(y, ((0, 0), (0, -k % 128))).reshape(n, -1, 128)


def quant(y: np.ndarray):
    """(codes as numbers N x K, exponents N x blocks) of finite y."""
    b = blocks(y)
    e = scale_exp(np.abs(b).max(2))
    return e4m3(b * 2.0 ** -e[:, :, None]).reshape(y.shape[0], -1)[:, :y.shape[1]], e


def check_codes(codes: torch.Tensor, scales: torch.Tensor, y: np.ndarray, delta: float):
    """Codes and scales of values that are within a factor 1 +- delta of y: each scale is one that such a largest
    magnitude gives, each code one that such a value gives at that scale."""
    b = blocks(y)
    amax = np.abs(b).max(2)
    e = scales.cpu().view(torch.uint8).numpy().astype(np.float64) - 127
    assert ((e == scale_exp(amax * (1 - delta))) | (e == scale_exp(amax * (1 + delta)))).all()
    v = np.abs(b) * 2.0 ** -e[:, :, None]
    got = blocks(f64(codes))
    assert (e4m3(v * (1 - delta)) <= np.abs(got)).all() and (np.abs(got) <= e4m3(v * (1 + delta))).all()
    assert ((np.sign(got) == np.sign(b)) | (got == 0)).all()


def values_of(codes: torch.Tensor, scales: torch.Tensor) -> np.ndarray:
    """Codes (N x K) with their scales (N x blocks), as numbers."""
    s = 2.0 ** (scales.cpu().view(torch.uint8).numpy().astype(np.float64) - 127)
    return f64(codes) * np.repeat(s, 128, 1)[:, :codes.shape[1]]


def norm(h: np.ndarray, gamma: np.ndarray, eps: float):
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * gamma, rstd


def norm_back(dy, h, rstd, gamma, dh):
    xhat = h * rstd[:, None]
    g = gamma * dy
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * xhat).sum(0)


def keep2(w: np.ndarray) -> np.ndarray:
    """2:4 pattern (M x K bool): of each four, those beaten by at most one other; lower index wins ties."""
    m, k = w.shape
    a = np.abs(w).reshape(m, k // 4, 4)
    beaten = np.zeros(a.shape, int)
    for t in range(4):
        for u in range(4):
            if u != t:
                beaten[:, :, t] += (a[:, :, u] > a[:, :, t]) | ((a[:, :, u] == a[:, :, t]) & (u < t))
    return (beaten < 2).reshape(m, k)


def weight(w: np.ndarray, kept: np.ndarray) -> np.ndarray:
    """What an M x K weight reads as after pruning and coding with a scale for each 128 x 128 block."""
    m, k = w.shape
    p = np.pad(w * kept, ((0, -m % 128), (0, -k % 128)))
    b = p.reshape(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    s = 2.0 ** scale_exp(np.abs(b).max((1, 3)))[:, None, :, None]
    return (e4m3(b / s) * s).reshape(p.shape)[:m, :k]
