"""Binding of the layer operators (include/sp24_layer.h): the 2:4 products with bias, activation and residual in their
epilogue, that epilogue's gradient, and an AdamW step over many tensors.

The functions have the C entry points' names and only marshal arguments, in _layer_binding.so (binding/layer_binding.cpp),
allocate outputs that are not given, and hold the workspaces (torch tensors, released to the caching allocator in stream
order)."""
from __future__ import annotations

import ctypes
import os

import torch

from . import SP24_ACT_GELU, SP24_ACT_NONE, SP24_ACT_RELU, SP24_ACT_SILU, _check, _layout, load_library

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_layer_binding.so")
_ACTIVATIONS = {"none": SP24_ACT_NONE, "gelu": SP24_ACT_GELU, "relu": SP24_ACT_RELU, "silu": SP24_ACT_SILU}
_native = None


def _load_native():
    """The extension module, built with libsp24.so; loaded at the first call. Raises if it is missing."""
    global _native
    load_library()
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is not built; run `python -m structured_sparse_gemm_sp24_amd.build` "
                           "(there is no fallback path)")
    from . import _layer_binding
    _layer_binding.init(_check, torch._C._cuda_getCurrentRawStream)
    _native = _layer_binding
    return _native


def bind(lib: ctypes.CDLL) -> None:
    """Argument types of the entry points of include/sp24_layer.h."""
    P, I64, I, D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
    lib.sp24_gemm_bf16_fused.argtypes = [P, P, I64, I64, P, I64, I64, I64, P, I, P, I64, I64, P, I64, I64, P, I, I64, I64, I64, I, P]
    lib.sp24_gemm_fp8_fused.argtypes = [P, P, P, I64, I64, P, I64, I64, P, I64, P, I, P, I64, P, I64, P, I, I64, P]
    lib.sp24_epilogue_backward_bytes.argtypes = [I64, I64, ctypes.POINTER(I64)]
    lib.sp24_epilogue_backward.argtypes = [P, I, I64, I64, I64, P, I64, I, P, I64, P, P, P]
    lib.sp24_adamw.argtypes = [P, I64, I, I, I, D, P, I64, P, D, D, D, D, P, ctypes.c_uint64, P, P]


def _activation(name) -> int:
    if name in _ACTIVATIONS:
        return _ACTIVATIONS[name]
    if name in _ACTIVATIONS.values():
        return name
    raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}, not {name!r}")


def sp24_gemm_bf16_fused(values: torch.Tensor, meta: torch.Tensor, M: int, X: torch.Tensor, bias: torch.Tensor | None = None,
                         activation="none", residual: torch.Tensor | None = None, preact=None, layout="feature",
                         out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None):
    """Y = act(W X + bias) + residual for a 2:4 weight in bf16, layouts and batches as sp24_gemm_bf16_ex. activation: "none",
    "gelu", "relu" or "silu"; bias fp32[M]; residual of Y's type and shape (give it as ``out`` too to add in place; a batch
    may share one through a stride of 0). With ``preact`` (True, or a tensor to fill) returns (Y, Z), Z = W X + bias
    rounded to Y's type: what sp24_epilogue_backward needs, token-major (feature-major it gives dZ alone). A batch's entries
    lie on 16 bytes: where their size is no multiple of that, give ``out`` (and ``preact``) with strides that are."""
    return (_native or _load_native()).gemm_bf16(values, meta, M, X, bias, _activation(activation), residual, preact, _layout(layout), out_dtype, out)


def sp24_gemm_fp8_fused(values: torch.Tensor, meta: torch.Tensor, w_scales: torch.Tensor, M: int, X: torch.Tensor,
                        x_scales: torch.Tensor, bias: torch.Tensor | None = None, activation="none",
                        residual: torch.Tensor | None = None, preact=None, out_dtype: torch.dtype = torch.bfloat16,
                        out: torch.Tensor | None = None):
    """Y (N x M, bf16 or fp16) = act(X W^T + bias) + residual for operands as sp24_gemm_fp8 takes them, the rest as
    sp24_gemm_bf16_fused."""
    return (_native or _load_native()).gemm_fp8(values, meta, w_scales, M, X, x_scales, bias, _activation(activation), residual, preact, out_dtype, out)


def sp24_epilogue_backward(dY: torch.Tensor, preact: torch.Tensor | None = None, activation="none", dZ: torch.Tensor | None = None,
                           dbias: torch.Tensor | None = None, want_dbias: bool = True):
    """Gradients of the products' epilogue (token-major): (dZ, dbias) with dZ = dY act'(preact) of dY's type, what the weight's
    and the input's gradients take, and dbias its sum over tokens (fp32[M]; None with want_dbias=False and no ``dbias``).
    ``dZ`` may be dY or preact. Without an activation dZ is dY itself. The residual's gradient is dY. Of feature-major
    matrices, an entry of a batch a call, take dZ with want_dbias=False: the sum that dbias holds would be one over channels."""
    return (_native or _load_native()).epilogue_backward(dY, preact, _activation(activation), dZ, dbias, bool(want_dbias))


def sp24_adamw_state(param: torch.Tensor, bits: int = 32) -> tuple:
    """A parameter's moments before its first step: (m, v) in fp32, or with bits=8 (m codes e4m3, m scales, v codes uint8, v
    scales): for each 128 consecutive elements m = code * scale and v = (code * scale)^2."""
    if bits == 32:
        return torch.zeros_like(param, dtype=torch.float32), torch.zeros_like(param, dtype=torch.float32)
    if bits != 8:
        raise ValueError(f"bits must be 8 or 32, not {bits}")
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device=param.device)  # noqa: E731
    blocks = (param.numel() + 127) // 128
    return (zeros(param.shape).view(torch.float8_e4m3fn), zeros(blocks).view(torch.float8_e8m0fnu),
            zeros(param.shape), zeros(blocks).view(torch.float8_e8m0fnu))


def sp24_adamw(params, grads, states, step, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: torch.Tensor | None = None, seed: int = 0, copies=None, out=None, first_index: int = 0) -> None:
    """One step of AdamW over a list of fp32 parameters (contiguous, on one device), in place: grads of one 16- or 32-bit type
    (None passes a parameter over, and its places in ``copies`` and ``out``), states from sp24_adamw_state, of one kind. ``step`` counts from 1; it and ``lr`` may be
    device tensors (int64 and fp32) that are read when the kernels run, as a captured graph needs. ``grad_scale`` (a device fp32)
    multiplies the gradients. ``copies``: bf16 or fp16 tensors (or None) that receive the new weights rounded. ``seed``: of the
    random rounding of 8-bit states, which also takes the parameter's place in the model: ``first_index`` is that of params[0], so
    that groups of parameters with a call each round independently. ``out``: (parameters, states) to write to instead."""
    params_out, states_out = (None, None) if out is None else out
    (_native or _load_native()).adamw(params, grads, states, step, lr, betas[0], betas[1], eps, weight_decay, grad_scale, seed, copies,
                                      params_out, states_out, first_index)
