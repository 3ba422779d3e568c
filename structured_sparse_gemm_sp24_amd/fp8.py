"""Binding of the 8-bit floating-point operators (include/sp24_fp8.h): activations as e4m3 codes with an e8m0 scale
for each 128 channels of a token, 2:4 weights as e4m3 values with a scale for each 128 x 128 block.

The functions have the C entry points' names and only marshal arguments, allocate outputs that are not given, and
hold the workspaces (torch tensors, released to the caching allocator in stream order)."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _TORCH_TO_SP24, SP24_SCORE_MAGNITUDE, _check, load_library

CODES, SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)
# These calls are a few microseconds of device work at one token, so their host side is kept short: the current
# stream's handle without a Stream object, and outputs from the allocator's direct entry (0.7 us against 1.6 us for
# torch.empty), both on the current device, which _on_device makes the operands'.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty_strided = torch._C._dynamo.guards._empty_strided_cuda


def bind(lib: ctypes.CDLL) -> None:
    """Argument types of the entry points of include/sp24_fp8.h."""
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    lib.sp24_quant_fp8.argtypes = [P, I, I64, I64, I64, P, I64, P, I64, P]
    lib.sp24_rmsnorm_fp8.argtypes = [P, I, I64, I64, I64, P, I64, P, F, P, I64, P, I64, P, I64, P, P]
    lib.sp24_rmsnorm_backward_bytes.argtypes = [I64, I64, ctypes.POINTER(I64)]
    lib.sp24_rmsnorm_backward.argtypes = [P, I, I64, I64, I64, P, I64, P, P, P, I64, P, I64, P, P, P]
    lib.sp24_prune_compress_fp8.argtypes = [P, I, I64, I64, I64, I, P, P, P, P, P]
    lib.sp24_decompress_fp8.argtypes = [P, P, P, I64, I64, P, I, I64, P]
    lib.sp24_gemm_fp8.argtypes = [P, P, P, I64, I64, P, I64, I64, P, I64, P, I, I64, P]
    lib.sp24_grad_weight_fp8_bytes.argtypes = [I64, I64, I64, ctypes.POINTER(I64)]
    lib.sp24_grad_weight_fp8.argtypes = [P, I64, I64, I64, P, I64, I64, P, I64, P, P, I, I64, P, P]


def _on_device(fn):
    """Runs fn on its first operand's device, a GPU."""
    @functools.wraps(fn)
    def call(first, *args, **kw):
        if not first.is_cuda:
            raise ValueError("sp24 operates on device tensors only")
        if first.get_device() == _current_device():
            return fn(first, *args, **kw)
        with torch.cuda.device(first.device):
            return fn(first, *args, **kw)
    return call


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _bad(t: torch.Tensor, name: str, dev: int, dtype, shape) -> None:
    """Says what is wrong with an operand that _matrix or _vector has refused."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the first operand's device")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be of type {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must have unit stride along its last dimension")


def _matrix(t: torch.Tensor, name: str, dev: int, dtype: torch.dtype, rows: int, cols: int) -> int:
    """Checks a row-major matrix and returns its row pitch in elements (of a single row, which has none, its length
    rounded up to what every entry point takes)."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, cols):
        _bad(t, name, dev, dtype, (rows, cols))
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        _bad(t, name, dev, dtype, (rows, cols))
    return s0 if rows > 1 else (cols + 15) // 16 * 16


def _first(t: torch.Tensor, name: str, dtypes) -> tuple:
    """(device index, rows, columns, row pitch) of the operand that the others are checked against."""
    if t.dtype not in dtypes or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix of one of the types {dtypes}, not {t.dtype} {tuple(t.shape)}")
    rows, cols = t.shape
    dev = t.get_device()
    return dev, rows, cols, _matrix(t, name, dev, t.dtype, rows, cols)


def _vector(t: torch.Tensor, name: str, dev: int, dtype: torch.dtype, n: int) -> int:
    """Checks a contiguous vector and returns its address."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        _bad(t, name, dev, dtype, (n,))
    return t.data_ptr()


def _out(t, name: str, dev: int, dtype: torch.dtype, rows: int, cols: int):
    """(tensor, pitch) of an output matrix, made here when it is not given."""
    if t is None:
        return _empty_strided((rows, cols), (cols, 1), dtype), cols
    return t, _matrix(t, name, dev, dtype, rows, cols)


def _weight(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, K: int, dev: int) -> None:
    """Checks a compressed weight's buffers (sizes as sp24_compressed_bytes)."""
    kb = _blocks(K)
    tiles = (M + 15) // 16 * kb
    _vector(values, "values", dev, CODES, 1024 * tiles)
    _vector(meta, "meta", dev, torch.uint8, 256 * tiles)
    if _matrix(w_scales, "w_scales", dev, SCALES, _blocks(M), kb) != kb and w_scales.shape[0] > 1:
        raise ValueError("w_scales must be contiguous")


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name: str, *sizes: int) -> int:
    n = ctypes.c_int64()
    _check(name, getattr(load_library(), name)(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(name: str, *sizes: int):
    """A workspace of the size that the entry point `name` gives, or None."""
    n = _workspace_bytes(name, *sizes)
    return _empty_strided((n,), (1,), torch.uint8) if n else None


def _ptr(t):
    return None if t is None else t.data_ptr()


@_on_device
def sp24_quant_fp8(X: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """X (N x K, bf16, fp16 or fp32) as (codes, scales): e4m3 N x K, and e8m0 N x ceil(K / 128)."""
    dev, N, K, ldx = _first(X, "X", _FLOATS)
    codes, ldc = _out(codes, "codes", dev, CODES, N, K)
    scales, lds = _out(scales, "scales", dev, SCALES, N, _blocks(K))
    _check("sp24_quant_fp8", load_library().sp24_quant_fp8(
        X.data_ptr(), _TORCH_TO_SP24[X.dtype], N, K, ldx, codes.data_ptr(), ldc, scales.data_ptr(), lds, _raw_stream(dev)))
    return codes, scales


@_on_device
def sp24_rmsnorm_fp8(X: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                     H: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """Root-mean-square norm of X (+ residual) as 8-bit codes: returns (codes, scales, H, rstd). H is X + residual
    rounded to X's type (give X or residual itself to update it in place), X where there is no residual; rstd
    (fp32[N]) is what sp24_rmsnorm_backward needs beside H."""
    dev, N, K, ldx = _first(X, "X", _FLOATS)
    dt = X.dtype
    g = _vector(gamma, "gamma", dev, dt, K)
    codes, ldc = _out(codes, "codes", dev, CODES, N, K)
    scales, lds = _out(scales, "scales", dev, SCALES, N, _blocks(K))
    if rstd is None:
        rstd = _empty_strided((N,), (1,), torch.float32)
    else:
        _vector(rstd, "rstd", dev, torch.float32, N)
    if residual is None:
        if H is not None:
            raise ValueError("H is only written with a residual")
        r, ldr, h, ldh = None, 0, None, 0
        H = X
    else:
        ldr = _matrix(residual, "residual", dev, dt, N, K)
        H, ldh = _out(H, "H", dev, dt, N, K)
        r, h = residual.data_ptr(), H.data_ptr()
    _check("sp24_rmsnorm_fp8", load_library().sp24_rmsnorm_fp8(
        X.data_ptr(), _TORCH_TO_SP24[dt], N, K, ldx, r, ldr, g, eps, h, ldh, codes.data_ptr(), ldc, scales.data_ptr(), lds,
        rstd.data_ptr(), _raw_stream(dev)))
    return codes, scales, H, rstd


@_on_device
def sp24_rmsnorm_backward(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor,
                          dH: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                          dgamma: torch.Tensor | None = None):
    """Gradients of the norm: (dX, dgamma), dX of H's type (the gradient of X and of the residual alike, with dH, the
    residual stream's own gradient, added), dgamma fp32[K]. H and rstd are what sp24_rmsnorm_fp8 returned."""
    dev, N, K, ldh = _first(H, "H", _FLOATS)
    dt = H.dtype
    lddy = _matrix(dY, "dY", dev, dt, N, K)
    g = _vector(gamma, "gamma", dev, dt, K)
    r = _vector(rstd, "rstd", dev, torch.float32, N)
    dh, lddh = (None, 0) if dH is None else (dH.data_ptr(), _matrix(dH, "dH", dev, dt, N, K))
    dX, lddx = _out(dX, "dX", dev, dt, N, K)
    if dgamma is None:
        dgamma = _empty_strided((K,), (1,), torch.float32)
    else:
        _vector(dgamma, "dgamma", dev, torch.float32, K)
    work = _workspace("sp24_rmsnorm_backward_bytes", N, K)
    _check("sp24_rmsnorm_backward", load_library().sp24_rmsnorm_backward(
        dY.data_ptr(), _TORCH_TO_SP24[dt], N, K, lddy, H.data_ptr(), ldh, r, g, dh, lddh, dX.data_ptr(), lddx,
        dgamma.data_ptr(), work.data_ptr(), _raw_stream(dev)))
    return dX, dgamma


@_on_device
def sp24_prune_compress_fp8(W: torch.Tensor, score: int = SP24_SCORE_MAGNITUDE, norms: torch.Tensor | None = None):
    """2:4 prune + compress of W (M x K) to 8 bits: (values, meta, w_scales), 1-D e4m3 values and uint8 metadata in
    the tiled layout, and e8m0 scales ceil(M / 128) x ceil(K / 128)."""
    dev, M, K, ldw = _first(W, "W", _FLOATS)
    if norms is not None:
        _vector(norms, "norms", dev, torch.float32, K)
    tiles = (M + 15) // 16 * _blocks(K)
    values = torch.empty(1024 * tiles, dtype=CODES, device=W.device)
    meta = torch.empty(256 * tiles, dtype=torch.uint8, device=W.device)
    w_scales = torch.empty((_blocks(M), _blocks(K)), dtype=SCALES, device=W.device)
    _check("sp24_prune_compress_fp8", load_library().sp24_prune_compress_fp8(
        W.data_ptr(), _TORCH_TO_SP24[W.dtype], M, K, ldw, int(score), _ptr(norms), values.data_ptr(), meta.data_ptr(),
        w_scales.data_ptr(), _raw_stream(dev)))
    return values, meta, w_scales


@_on_device
def sp24_decompress_fp8(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, K: int,
                        out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The dense M x K weight (bf16 or fp32), +0 at pruned places: dX = dY @ it is the input's gradient."""
    dev = values.get_device()
    _weight(values, meta, w_scales, M, K, dev)
    out, ldw = _out(out, "out", dev, out_dtype if out is None else out.dtype, M, K)
    _check("sp24_decompress_fp8", load_library().sp24_decompress_fp8(
        values.data_ptr(), meta.data_ptr(), w_scales.data_ptr(), M, K, out.data_ptr(), _TORCH_TO_SP24.get(out.dtype, -1),
        ldw, _raw_stream(dev)))
    return out


@_on_device
def sp24_gemm_fp8(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, X: torch.Tensor,
                  x_scales: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Y (N x M, bf16 or fp16) = X W^T for a 2:4 weight in 8 bits and X (N x K) as codes and scales."""
    dev, N, K, ldx = _first(X, "X", (CODES,))
    lds = _matrix(x_scales, "x_scales", dev, SCALES, N, _blocks(K))
    _weight(values, meta, w_scales, M, K, dev)
    out, ldy = _out(out, "out", dev, out_dtype if out is None else out.dtype, N, M)
    _check("sp24_gemm_fp8", load_library().sp24_gemm_fp8(
        values.data_ptr(), meta.data_ptr(), w_scales.data_ptr(), M, K, X.data_ptr(), N, ldx, x_scales.data_ptr(), lds,
        out.data_ptr(), _TORCH_TO_SP24.get(out.dtype, -1), ldy, _raw_stream(dev)))
    return out


@_on_device
def sp24_grad_weight_fp8(dY: torch.Tensor, X: torch.Tensor, x_scales: torch.Tensor, meta: torch.Tensor | None = None,
                         out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """dW (M x K, fp32 or bf16) = dY^T X from bf16 dY (N x M) and the 8-bit copy of X (N x K codes, scales). With the
    weight's metadata (``meta``) dW is zero at its pruned places."""
    dev, N, M, lddy = _first(dY, "dY", (torch.bfloat16,))
    K = X.shape[-1]
    ldx = _matrix(X, "X", dev, CODES, N, K)
    lds = _matrix(x_scales, "x_scales", dev, SCALES, N, _blocks(K))
    if meta is not None:
        _vector(meta, "meta", dev, torch.uint8, 256 * ((M + 15) // 16) * _blocks(K))
    out, ldw = _out(out, "out", dev, out_dtype if out is None else out.dtype, M, K)
    work = _workspace("sp24_grad_weight_fp8_bytes", M, K, N)
    _check("sp24_grad_weight_fp8", load_library().sp24_grad_weight_fp8(
        dY.data_ptr(), N, M, lddy, X.data_ptr(), K, ldx, x_scales.data_ptr(), lds, _ptr(meta), out.data_ptr(),
        _TORCH_TO_SP24.get(out.dtype, -1), ldw, _ptr(work), _raw_stream(dev)))
    return out
