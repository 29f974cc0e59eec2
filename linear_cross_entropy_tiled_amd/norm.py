"""Layer norm of hidden states: the torch side of flce_layer_norm_* (include/flce.h has the formulas).  The autograd
node is C++ (csrc/flce_torch.cpp)."""
from __future__ import annotations

import functools
import math

from . import DTYPES, _dtype_name, between_graphs, flce_layer_norm_workspace_size, flce_norm_params, torch_ops
from .logprobs import has_tangent


def rows_apart(t):
    """Whether rows are contiguous and do not overlap; only the distance between them is free."""
    return t.is_contiguous() or ((t.stride(1) == 1 or t.shape[1] == 1)
                                 and (t.stride(0) >= t.shape[1] or t.shape[0] == 1))


def row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


@functools.lru_cache(maxsize=1024)
def _workspace(rows, cols, ld_x, dtype, param_dtype, eps):
    """Bytes of the backward's workspace; refuses what the C entry points would."""
    return flce_layer_norm_workspace_size(flce_norm_params(rows, cols, ld_x, 0, dtype, param_dtype, eps, 0))


def _check_vector(t, name, x, h):
    import torch
    if t.dtype != x.dtype and t.dtype != torch.float32:
        raise TypeError(f"{name} must be {x.dtype} as x, or float32, not {t.dtype}")
    if t.dim() != 1 or t.shape[0] != h:
        raise ValueError(f"{name} must have shape ({h},), got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check(x, weight, bias, eps):
    """Types, shapes, layout and device.  The kernels trust all of them.  Returns the backward's workspace size."""
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    dtype = param_dtype = DTYPES[_dtype_name(x)]
    n, h = x.shape
    if h < 1:
        raise ValueError("rows must hold at least one value")
    if weight is not None:
        _check_vector(weight, "weight", x, h)
        if weight.dtype != x.dtype:
            param_dtype = DTYPES["f32"]
    if bias is not None:
        _check_vector(bias, "bias", x, h)
        if weight is not None and bias.dtype != weight.dtype:
            raise TypeError(f"bias dtype {bias.dtype} differs from weight's {weight.dtype}")
        if bias.dtype != x.dtype:
            param_dtype = DTYPES["f32"]
    if not rows_apart(x):
        raise ValueError(f"x must have contiguous rows that do not overlap, got strides {x.stride()}")
    if not (math.isfinite(eps) and eps >= 0):
        raise ValueError(f"eps must be at least 0, got {eps}")
    dev = x.device
    for name, t in (("x", x), ("weight", weight), ("bias", bias)):
        if t is not None and (not t.is_cuda or t.device != dev):
            raise ValueError(f"{name} must be on x's GPU ({dev}), not {t.device}")
    return _workspace(n, h, row_stride(x), dtype, param_dtype, eps)


@functools.lru_cache(maxsize=None)
def _op():
    return torch_ops()._layer_norm.default


@between_graphs
def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5):
    """Layer norm of the rows of x (N, H): weight (x - mean) / sqrt(var + eps) + bias, in x's dtype (fp32, bf16,
    fp16), formed in fp32.  Differentiable in x, weight and bias.

    weight and bias (H,) are of x's dtype or both fp32; without them ones and zeros.  Rows of x are contiguous, at
    any distance.  H may be any size up to 2^20; rows of whole 16-byte pieces run faster."""
    eps = float(eps)
    workspace = _check(x, weight, bias, eps)
    if has_tangent(x, weight, bias):
        raise NotImplementedError("layer_norm has no forward-mode derivative")
    return _op()(x, weight, bias, eps, workspace)
