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


def _check(x, weight, bias, eps):
    import torch
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    _dtype_name(x)
    h = x.shape[1]
    if h < 1:
        raise ValueError("rows must hold at least one value")
    kind = None
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        if t.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"{name} must be {x.dtype} as x, or float32, not {t.dtype}")
        if kind is not None and t.dtype != kind:
            raise TypeError(f"bias dtype {t.dtype} differs from weight's {kind}")
        kind = t.dtype
        if t.dim() != 1 or t.shape[0] != h:
            raise ValueError(f"{name} must have shape ({h},), got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not rows_apart(x):
        raise ValueError(f"x must have contiguous rows that do not overlap, got strides {x.stride()}")
    if not (math.isfinite(eps) and eps >= 0):
        raise ValueError(f"eps must be at least 0, got {eps}")
    for name, t in (("x", x), ("weight", weight), ("bias", bias)):
        if t is not None and (t.device.type != "cuda" or t.device != x.device):
            raise ValueError(f"{name} must be on x's GPU ({x.device}), not {t.device}")
    dtype = DTYPES[_dtype_name(x)]
    return flce_norm_params(x.shape[0], h, row_stride(x), 0, dtype,
                            DTYPES["f32"] if kind == torch.float32 else dtype, eps, 0)


def _forward(p, x, weight, bias, keep):
    import torch
    dev = x.device
    with on_device(dev):
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        stats = torch.empty((2, x.shape[0]), dtype=torch.float32, device=dev) if keep else None
        at = _ptr(stats)
        raise_for(flce_layer_norm_forward(p, _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), at,
                                          at + 4 * x.shape[0] if keep else None, stream_handle(dev)),
                  "flce_layer_norm_forward")
    return y, stats


@functools.lru_cache(maxsize=None)
def _function():
    import torch

    class LayerNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, p):
            y, stats = _forward(p, x, weight, bias, True)
            ctx.save_for_backward(x, weight, stats)
            ctx.p, ctx.bias_like = p, None if bias is None else bias.dtype
            return y

        @first_order
        def backward(ctx, g):
            x, weight, stats = ctx.saved_tensors
            if not rows_apart(g):
                g = g.contiguous()
            p, dev = ctx.p, x.device
            p = flce_norm_params(p.rows, p.cols, p.ld_x, row_stride(g), p.dtype, p.param_dtype, p.eps, 0)
            need = ctx.needs_input_grad
            with on_device(dev):
                gx = torch.empty(x.shape, dtype=x.dtype, device=dev) if need[0] else None
                gw = torch.empty_like(weight) if need[1] else None
                gb = torch.empty(x.shape[1], dtype=ctx.bias_like, device=dev) if need[2] else None
                ws_bytes = flce_layer_norm_workspace_size(p) if need[1] or need[2] else 0
                workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
                at = _ptr(stats)
                raise_for(flce_layer_norm_backward(p, _ptr(x), _ptr(weight), at, at + 4 * x.shape[0], _ptr(g),
                                                   _ptr(gx), _ptr(gw), _ptr(gb), _ptr(workspace), ws_bytes,
                                                   stream_handle(dev)), "flce_layer_norm_backward")
            return gx, gw, gb, None

    return LayerNorm


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5):
    """Layer norm of the rows of x (N, H): weight (x - mean) / sqrt(var + eps) + bias, in x's dtype (fp32, bf16,
    fp16), formed in fp32.  Differentiable in x, weight and bias.

    weight and bias (H,) are of x's dtype or both fp32; without them ones and zeros.  Rows of x are contiguous, at
    any distance.  H may be any size up to 2^20; rows of whole 16-byte pieces run faster."""
    p = _check(x, weight, bias, eps)
    if differentiable(x, weight, bias):
        return _function().apply(x, weight, bias, p)
    return _forward(p, x, weight, bias, False)[0]
