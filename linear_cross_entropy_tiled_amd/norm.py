"""Layer norm of hidden states: the torch side of flce_layer_norm_* (include/flce.h has the formulas)."""
from __future__ import annotations

import functools
import math

from . import (DTYPES, _dtype_name, _ptr, flce_layer_norm_backward, flce_layer_norm_forward,
               flce_layer_norm_workspace_size, flce_norm_params)
from .logprobs import differentiable, first_order, on_device, raise_for, stream_handle


def rows_apart(t):
    """Whether rows are contiguous and do not overlap; only the distance between them is free."""
    return t.is_contiguous() or ((t.stride(1) == 1 or t.shape[1] == 1)
                                 and (t.stride(0) >= t.shape[1] or t.shape[0] == 1))


def row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


@functools.lru_cache(maxsize=1024)
def _params(rows, cols, ld_x, ld_grad, dtype, param_dtype, eps):
    return flce_norm_params(rows, cols, ld_x, ld_grad, dtype, param_dtype, eps, 0)


@functools.lru_cache(maxsize=1024)
def _workspace(rows, cols):
    return flce_layer_norm_workspace_size(flce_norm_params(rows, cols, 0, 0, 0, 0, 0.0, 0))


def _check_vector(t, name, x, h):
    import torch
    if t.dtype != x.dtype and t.dtype != torch.float32:
        raise TypeError(f"{name} must be {x.dtype} as x, or float32, not {t.dtype}")
    if t.dim() != 1 or t.shape[0] != h:
        raise ValueError(f"{name} must have shape ({h},), got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check(x, weight, bias, eps):
    """Types, shapes, layout and device.  The kernels trust all of them.  Returns the call's parameters."""
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
    return _params(n, h, row_stride(x), 0, dtype, param_dtype, eps)


def _forward(p, x, weight, bias, keep):
    import torch
    dev = x.device
    with on_device(dev):
        y = x.new_empty(x.shape)
        stats = torch.empty((2, p.rows), dtype=torch.float32, device=dev) if keep else None
        at = _ptr(stats)
        raise_for(flce_layer_norm_forward(p, x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), at,
                                          at + 4 * p.rows if keep else None, stream_handle(dev)),
                  "flce_layer_norm_forward")
    return y, stats


@functools.lru_cache(maxsize=None)
def _function():
    import torch

    class LayerNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, p):
            y, stats = _forward(p, x, weight, bias, True)
            ctx.save_for_backward(x, weight, bias, stats)
            ctx.p = p
            return y

        @first_order
        def backward(ctx, g):
            x, weight, bias, stats = ctx.saved_tensors
            p, dev = ctx.p, x.device
            if not g.is_contiguous():
                if rows_apart(g):
                    p = _params(p.rows, p.cols, p.ld_x, row_stride(g), p.dtype, p.param_dtype, p.eps)
                else:
                    g = g.contiguous()
            need_x, need_w, need_b, _ = ctx.needs_input_grad
            with on_device(dev):
                gx = x.new_empty(x.shape) if need_x else None
                gw = torch.empty_like(weight) if need_w else None
                gb = torch.empty_like(bias) if need_b else None
                ws_bytes = _workspace(p.rows, p.cols) if need_w or need_b else 0
                workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
                at = stats.data_ptr()
                raise_for(flce_layer_norm_backward(p, x.data_ptr(), _ptr(weight), at, at + 4 * p.rows, g.data_ptr(),
                                                   _ptr(gx), _ptr(gw), _ptr(gb), _ptr(workspace), ws_bytes,
                                                   stream_handle(dev)), "flce_layer_norm_backward")
            return gx, gw, gb, None

    return LayerNorm


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5):
    """Layer norm of the rows of x (N, H): weight (x - mean) / sqrt(var + eps) + bias, in x's dtype (fp32, bf16,
    fp16), formed in fp32.  Differentiable in x, weight and bias.

    weight and bias (H,) are of x's dtype or both fp32; without them ones and zeros.  Rows of x are contiguous, at
    any distance.  H may be any size up to 2^20; rows of whole 16-byte pieces run faster."""
    p = _check(x, weight, bias, float(eps))
    if differentiable(x, weight, bias):
        return _function().apply(x, weight, bias, p)
    return _forward(p, x, weight, bias, False)[0]
