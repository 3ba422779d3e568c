"""Binding of the 8-bit floating-point operators (include/sp24_fp8.h): activations as e4m3 codes with an e8m0 scale
for each 128 channels of a token, 2:4 weights as e4m3 values with a scale for each 128 x 128 block.

The functions have the C entry points' names and only marshal arguments, allocate outputs that are not given, and
hold the workspaces (torch tensors, released to the caching allocator in stream order)."""
from __future__ import annotations

import ctypes

import torch

from . import _TORCH_TO_SP24, SP24_SCORE_MAGNITUDE, _check, _check_compressed, load_library, sp24_compressed_bytes

CODES, SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without making a Stream object


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


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _matrix(t: torch.Tensor, name: str, device: torch.device, dtype, shape=None) -> int:
    """Checks a row-major matrix and returns its row pitch in elements (of a single row, which has none, its length
    rounded up to what every entry point takes)."""
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on the device of the first operand, a GPU")
    if t.dtype != dtype if isinstance(dtype, torch.dtype) else t.dtype not in dtype:
        raise ValueError(f"{name} must be of type {dtype}, not {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {tuple(shape) if shape else '(rows, columns)'}, not {tuple(t.shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.stride(0) if rows > 1 else (cols + 15) // 16 * 16


def _vector(t: torch.Tensor, name: str, device: torch.device, dtype: torch.dtype, n: int) -> None:
    if t.device != device or t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} values of type {dtype} on {device}")


def _out(t, name: str, device, dtype, shape):
    """(tensor, pitch) of an output, made here when it is not given."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device), shape[1]
    return t, _matrix(t, name, device, dtype, torch.Size(shape))


def _call(name: str, device: torch.device, *args) -> None:
    fn = getattr(load_library(), name)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            _check(name, fn(*args, _raw_stream(device.index)))
    else:
        _check(name, fn(*args, _raw_stream(device.index)))


def _weight(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, K: int, device) -> None:
    if values.dtype != CODES or values.device != device or meta.device != device:
        raise ValueError(f"values must be {CODES} and, with meta, on {device}")
    _check_compressed(values, meta, M, K)
    _matrix(w_scales, "w_scales", device, SCALES, torch.Size((_blocks(M), _blocks(K))))
    if not w_scales.is_contiguous():
        raise ValueError("w_scales must be contiguous")


def sp24_quant_fp8(X: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """X (N x K, bf16, fp16 or fp32) as (codes, scales): e4m3 N x K, and e8m0 N x ceil(K / 128)."""
    dev = X.device
    ldx = _matrix(X, "X", dev, _FLOATS)
    N, K = X.shape
    codes, ldc = _out(codes, "codes", dev, CODES, (N, K))
    scales, lds = _out(scales, "scales", dev, SCALES, (N, _blocks(K)))
    _call("sp24_quant_fp8", dev, X.data_ptr(), _TORCH_TO_SP24[X.dtype], N, K, ldx, codes.data_ptr(), ldc,
          scales.data_ptr(), lds)
    return codes, scales


def sp24_rmsnorm_fp8(X: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                     H: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """Root-mean-square norm of X (+ residual) as 8-bit codes: returns (codes, scales, H, rstd). H is X + residual
    rounded to X's type (give X or residual itself to update it in place), X where there is no residual; rstd
    (fp32[N]) is what sp24_rmsnorm_backward needs beside H."""
    dev, dt = X.device, X.dtype
    ldx = _matrix(X, "X", dev, _FLOATS)
    N, K = X.shape
    _vector(gamma, "gamma", dev, dt, K)
    codes, ldc = _out(codes, "codes", dev, CODES, (N, K))
    scales, lds = _out(scales, "scales", dev, SCALES, (N, _blocks(K)))
    if rstd is None:
        rstd = torch.empty(N, dtype=torch.float32, device=dev)
    else:
        _vector(rstd, "rstd", dev, torch.float32, N)
    if residual is None:
        if H is not None:
            raise ValueError("H is only written with a residual")
        r, ldr, h, ldh = None, 0, None, 0
    else:
        ldr = _matrix(residual, "residual", dev, dt, X.shape)
        H, ldh = _out(H, "H", dev, dt, (N, K))
        r, h = residual.data_ptr(), H.data_ptr()
    _call("sp24_rmsnorm_fp8", dev, X.data_ptr(), _TORCH_TO_SP24[dt], N, K, ldx, r, ldr, gamma.data_ptr(), eps, h, ldh,
          codes.data_ptr(), ldc, scales.data_ptr(), lds, rstd.data_ptr())
    return codes, scales, X if H is None else H, rstd


def sp24_rmsnorm_backward(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor,
                          dH: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                          dgamma: torch.Tensor | None = None):
    """Gradients of the norm: (dX, dgamma), dX of H's type (the gradient of X and of the residual alike, with dH, the
    residual stream's own gradient, added), dgamma fp32[K]. H and rstd are what sp24_rmsnorm_fp8 returned."""
    dev, dt = H.device, H.dtype
    ldh = _matrix(H, "H", dev, _FLOATS)
    N, K = H.shape
    lddy = _matrix(dY, "dY", dev, dt, H.shape)
    _vector(gamma, "gamma", dev, dt, K)
    _vector(rstd, "rstd", dev, torch.float32, N)
    dh, lddh = (None, 0) if dH is None else (dH.data_ptr(), _matrix(dH, "dH", dev, dt, H.shape))
    dX, lddx = _out(dX, "dX", dev, dt, (N, K))
    if dgamma is None:
        dgamma = torch.empty(K, dtype=torch.float32, device=dev)
    else:
        _vector(dgamma, "dgamma", dev, torch.float32, K)
    nb = ctypes.c_int64()
    _check("sp24_rmsnorm_backward_bytes", load_library().sp24_rmsnorm_backward_bytes(N, K, ctypes.byref(nb)))
    work = torch.empty(nb.value, dtype=torch.uint8, device=dev)
    _call("sp24_rmsnorm_backward", dev, dY.data_ptr(), _TORCH_TO_SP24[dt], N, K, lddy, H.data_ptr(), ldh,
          rstd.data_ptr(), gamma.data_ptr(), dh, lddh, dX.data_ptr(), lddx, dgamma.data_ptr(), work.data_ptr())
    return dX, dgamma


def sp24_prune_compress_fp8(W: torch.Tensor, score: int = SP24_SCORE_MAGNITUDE, norms: torch.Tensor | None = None):
    """2:4 prune + compress of W (M x K) to 8 bits: (values, meta, w_scales), 1-D e4m3 values and uint8 metadata in
    the tiled layout, and e8m0 scales ceil(M / 128) x ceil(K / 128)."""
    dev = W.device
    ldw = _matrix(W, "W", dev, _FLOATS)
    M, K = W.shape
    if norms is not None:
        _vector(norms, "norms", dev, torch.float32, K)
    vb, mb = sp24_compressed_bytes(M, K, CODES)
    values = torch.empty(vb, dtype=CODES, device=dev)
    meta = torch.empty(mb, dtype=torch.uint8, device=dev)
    w_scales = torch.empty((_blocks(M), _blocks(K)), dtype=SCALES, device=dev)
    _call("sp24_prune_compress_fp8", dev, W.data_ptr(), _TORCH_TO_SP24[W.dtype], M, K, ldw, int(score),
          None if norms is None else norms.data_ptr(), values.data_ptr(), meta.data_ptr(), w_scales.data_ptr())
    return values, meta, w_scales


def sp24_decompress_fp8(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, K: int,
                        out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The dense M x K weight (bf16 or fp32), +0 at pruned places: dX = dY @ it is the input's gradient."""
    dev = values.device
    _weight(values, meta, w_scales, M, K, dev)
    out, ldw = _out(out, "out", dev, out_dtype if out is None else out.dtype, (M, K))
    _call("sp24_decompress_fp8", dev, values.data_ptr(), meta.data_ptr(), w_scales.data_ptr(), M, K, out.data_ptr(),
          _TORCH_TO_SP24.get(out.dtype, -1), ldw)
    return out


def sp24_gemm_fp8(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, X: torch.Tensor,
                  x_scales: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Y (N x M, bf16 or fp16) = X W^T for a 2:4 weight in 8 bits and X (N x K) as codes and scales."""
    dev = X.device
    ldx = _matrix(X, "X", dev, CODES)
    N, K = X.shape
    lds = _matrix(x_scales, "x_scales", dev, SCALES, torch.Size((N, _blocks(K))))
    _weight(values, meta, w_scales, M, K, dev)
    out, ldy = _out(out, "out", dev, out_dtype if out is None else out.dtype, (N, M))
    _call("sp24_gemm_fp8", dev, values.data_ptr(), meta.data_ptr(), w_scales.data_ptr(), M, K, X.data_ptr(), N, ldx,
          x_scales.data_ptr(), lds, out.data_ptr(), _TORCH_TO_SP24.get(out.dtype, -1), ldy)
    return out


def sp24_grad_weight_fp8(dY: torch.Tensor, X: torch.Tensor, x_scales: torch.Tensor, meta: torch.Tensor | None = None,
                         out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """dW (M x K, fp32 or bf16) = dY^T X from bf16 dY (N x M) and the 8-bit copy of X (N x K codes, scales). With the
    weight's metadata (``meta``) dW is zero at its pruned places."""
    dev = X.device
    ldx = _matrix(X, "X", dev, CODES)
    N, K = X.shape
    lds = _matrix(x_scales, "x_scales", dev, SCALES, torch.Size((N, _blocks(K))))
    lddy = _matrix(dY, "dY", dev, torch.bfloat16)
    M = dY.shape[1]
    if dY.shape[0] != N:
        raise ValueError(f"dY has {dY.shape[0]} rows, X {N}")
    if meta is not None:
        _vector(meta, "meta", dev, torch.uint8, sp24_compressed_bytes(M, K, CODES)[1])
    out, ldw = _out(out, "out", dev, out_dtype if out is None else out.dtype, (M, K))
    nb = ctypes.c_int64()
    _check("sp24_grad_weight_fp8_bytes", load_library().sp24_grad_weight_fp8_bytes(M, K, N, ctypes.byref(nb)))
    work = torch.empty(nb.value, dtype=torch.uint8, device=dev) if nb.value else None
    _call("sp24_grad_weight_fp8", dev, dY.data_ptr(), N, M, lddy, X.data_ptr(), K, ldx, x_scales.data_ptr(), lds,
          None if meta is None else meta.data_ptr(), out.data_ptr(), _TORCH_TO_SP24.get(out.dtype, -1), ldw,
          None if work is None else work.data_ptr())
    return out
