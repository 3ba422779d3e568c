"""Binding of the 8-bit floating-point operators (include/sp24_fp8.h): activations as e4m3 codes with an e8m0 scale
for each 128 channels of a token, 2:4 weights as e4m3 values with a scale for each 128 x 128 block.

The functions have the C entry points' names and only marshal arguments, allocate outputs that are not given, and
hold the workspaces (torch tensors, released to the caching allocator in stream order). Those that a decoding or
training step calls do so in _fp8_binding.so (binding/fp8_binding.cpp): at one token they are a few microseconds of
device work, less than the same checks take in Python."""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

from . import _TORCH_TO_SP24, SP24_SCORE_MAGNITUDE, _check, load_library

CODES, SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_fp8_binding.so")
_raw_stream = torch._C._cuda_getCurrentRawStream
_native = None


def _load_native():
    """The extension module, built with libsp24.so; loaded at the first call. Raises if it is missing."""
    global _native
    load_library()
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is not built; run `python -m structured_sparse_gemm_sp24_amd.build` "
                           "(there is no fallback path)")
    from . import _fp8_binding
    _fp8_binding.init(_check, _raw_stream)
    _native = _fp8_binding
    return _native


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
    """Runs fn on its first operand's device, a GPU; that operand too may be given by its name."""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, **kw):
        if not args and name not in kw:
            raise TypeError(f"{fn.__name__}() needs {name}")
        first = args[0] if args else kw[name]
        if not first.is_cuda:
            raise ValueError("sp24 operates on device tensors only")
        with torch.cuda.device(first.device):
            return fn(*args, **kw)
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
        return torch.empty((rows, cols), dtype=dtype, device=f"cuda:{dev}"), cols
    return t, _matrix(t, name, dev, dtype, rows, cols)


def _weight(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, K: int, dev: int) -> None:
    """Checks a compressed weight's buffers (sizes as sp24_compressed_bytes)."""
    kb = _blocks(K)
    tiles = (M + 15) // 16 * kb
    _vector(values, "values", dev, CODES, 1024 * tiles)
    _vector(meta, "meta", dev, torch.uint8, 256 * tiles)
    if _matrix(w_scales, "w_scales", dev, SCALES, _blocks(M), kb) != kb and w_scales.shape[0] > 1:
        raise ValueError("w_scales must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def sp24_quant_fp8(X: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """X (N x K, bf16, fp16 or fp32) as (codes, scales): e4m3 N x K, and e8m0 N x ceil(K / 128)."""
    return (_native or _load_native()).quant(X, codes, scales)


def sp24_rmsnorm_fp8(X: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                     H: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """Root-mean-square norm of X (+ residual) as 8-bit codes: returns (codes, scales, H, rstd). H is X + residual
    rounded to X's type (give X or residual itself to update it in place), X where there is no residual; rstd
    (fp32[N]) is what sp24_rmsnorm_backward needs beside H."""
    return (_native or _load_native()).rmsnorm(X, gamma, eps, residual, H, codes, scales, rstd)


def sp24_rmsnorm_backward(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor,
                          dH: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                          dgamma: torch.Tensor | None = None):
    """Gradients of the norm: (dX, dgamma), dX of H's type (the gradient of X and of the residual alike, with dH, the
    residual stream's own gradient, added), dgamma fp32[K]. H and rstd are what sp24_rmsnorm_fp8 returned."""
    return (_native or _load_native()).rmsnorm_backward(dY, H, rstd, gamma, dH, dX, dgamma)


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


def sp24_gemm_fp8(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, X: torch.Tensor,
                  x_scales: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Y (N x M, bf16 or fp16) = X W^T for a 2:4 weight in 8 bits and X (N x K) as codes and scales."""
    return (_native or _load_native()).gemm(values, meta, w_scales, M, X, x_scales, out_dtype, out)


def sp24_grad_weight_fp8(dY: torch.Tensor, X: torch.Tensor, x_scales: torch.Tensor, meta: torch.Tensor | None = None,
                         out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """dW (M x K, fp32 or bf16) = dY^T X from bf16 dY (N x M) and the 8-bit copy of X (N x K codes, scales). With the
    weight's metadata (``meta``) dW is zero at its pruned places."""
    return (_native or _load_native()).grad_weight(dY, X, x_scales, meta, out_dtype, out)
