"""Per-token log-probabilities and entropies of a linear head: the torch side of
flce_logprobs_* (include/flce.h has the formulas)."""
from __future__ import annotations

import contextlib
import functools
from typing import Optional

from . import (DTYPES, FLCE_OK, FLCE_PASS_BACKWARD, FLCE_PASS_FORWARD, FlceError, _dtype_name, _ptr, _stream_handle,
               _targets_int32, _validate, between_graphs, by_pointers, flce_logprobs_backward, flce_logprobs_forward,
               flce_logprobs_int8, flce_logprobs_int8_workspace_size, flce_logprobs_mxfp4_workspace_size,
               flce_logprobs_workspace_size, flce_quantize_int8, make_params, torch_ops)


_SAME_DEVICE = contextlib.nullcontext()


def on_device(device):
    """The library launches on the current device: makes it the tensors'."""
    import torch
    # (current_device() asks the same after looking whether the runtime is up, which it is where there are tensors: 4 us
    # in a backward's thread)
    current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if device.index is None or device.index == current():
        return _SAME_DEVICE
    return torch.cuda.device(device)


def stream_handle(device):
    """The current stream of a GPU, without a torch.cuda.Stream object around it (3 us)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return _stream_handle(device) if raw is None or device.index is None else raw(device.index)


def differentiable(*tensors) -> bool:
    """Whether the call goes through its autograd function: autograd records it (without, the function's own cost
    is saved), or an input carries a forward-mode tangent, which the function refuses to drop."""
    import torch
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return True
    return has_tangent(*tensors)


def has_tangent(*tensors) -> bool:
    """Whether one of them is a dual tensor of forward-mode autograd (no_grad does not take tangents away)."""
    import torch
    ad = torch.autograd.forward_ad
    if getattr(ad, "_current_level", 0) < 0:       # no level is open: there are none (0.4 us a tensor saved)
        return False
    return any(t is not None and ad.unpack_dual(t).tangent is not None for t in tensors)


def first_order(backward):
    """backward for a torch.autograd.Function without a second derivative: once_differentiable, whose
    bookkeeping is skipped where autograd does not record the backward (small steps are bound by the
    Python that runs in the backward's thread)."""
    import torch
    from torch.autograd.function import once_differentiable
    recorded = once_differentiable(backward)

    def run(ctx, *grads):
        return recorded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)

    return staticmethod(run)


def upstream(g):
    """An upstream gradient as the kernels read it."""
    import torch
    return g if g is None or (g.dtype == torch.float32 and g.is_contiguous()) else g.to(torch.float32).contiguous()


def raise_for(rc, where):
    if rc != FLCE_OK:
        raise FlceError(rc, where)


def _forward(p, hidden, weight, bias, targets):
    import torch
    dev, n = hidden.device, hidden.shape[0]
    with on_device(dev):
        ws_bytes = flce_logprobs_workspace_size(p, FLCE_PASS_FORWARD)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        logps, entropy, lse = (torch.empty(n, dtype=torch.float32, device=dev) for _ in range(3))
        raise_for(flce_logprobs_forward(p, _ptr(hidden), _ptr(weight), _ptr(bias), _ptr(targets), _ptr(logps),
                                        _ptr(entropy), _ptr(lse), _ptr(workspace), ws_bytes, stream_handle(dev)),
                  "flce_logprobs_forward")
    return logps, entropy, lse


@functools.lru_cache(maxsize=None)
def _function():
    import torch

    class TokenLogprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, hidden, weight, bias, targets, p):
            logps, entropy, lse = _forward(p, hidden, weight, bias, targets)
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(hidden, weight, bias, targets, lse, entropy)
            ctx.p = p
            return logps, entropy

        @first_order
        def backward(ctx, g, h):
            if g is None and h is None:
                return (None,) * 5
            hidden, weight, bias, targets, lse, entropy = ctx.saved_tensors
            g, h = upstream(g), upstream(h)
            dev = hidden.device
            with on_device(dev):
                ws_bytes = flce_logprobs_workspace_size(ctx.p, FLCE_PASS_BACKWARD)
                workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
                gh, gw, gb = (torch.empty_like(t) if need else None     # a frozen head's are not computed
                              for t, need in zip((hidden, weight, bias), ctx.needs_input_grad))
                raise_for(flce_logprobs_backward(ctx.p, _ptr(hidden), _ptr(weight), _ptr(bias), _ptr(targets),
                                                 _ptr(lse), _ptr(entropy), _ptr(g), _ptr(h), _ptr(gh), _ptr(gw),
                                                 _ptr(gb), _ptr(workspace), ws_bytes, stream_handle(dev)),
                          "flce_logprobs_backward")
            return gh, gw, gb, None, None

    return TokenLogprobs


@by_pointers
def token_logprobs(hidden, weight, targets, bias=None, *, logit_scale: float = 1.0, softcap: Optional[float] = None,
                   ignore_index: int = -100, return_entropy: bool = False, vocab_chunk: int = 0):
    """Log-probabilities (N,) of ``targets`` under softmax(softcap(logit_scale (hidden @ weight.T + bias))),
    in fp32, without the (N, V) logits; with ``return_entropy`` also each row's entropy (nats).

    Both are differentiable in hidden, weight and bias (the backward recomputes the logit tiles).
    Rows whose target is ``ignore_index``, or no row of weight, give 0 and take no gradient.  ``vocab_chunk``: as in
    ``backward``.  hidden, weight and bias share one dtype (fp32, bf16, fp16)."""
    dt = _validate(hidden, weight, targets, bias, reduction="none")
    p = make_params(hidden.shape[0], hidden.shape[1], weight.shape[0], dtype=dt, logit_scale=logit_scale,
                    softcap=softcap, ignore_index=ignore_index, reduction="none",
                    targets_int32=_targets_int32(targets), vocab_chunk=vocab_chunk)
    if differentiable(hidden, weight, bias):
        logps, entropy = _function().apply(hidden, weight, bias, targets, p)
    else:
        logps, entropy, _ = _forward(p, hidden, weight, bias, targets)
    return (logps, entropy) if return_entropy else logps


# ----------------------------------------------------------------------------- 8-bit scoring

def _quantize(x):
    import torch
    dev = x.device
    with on_device(dev):
        q = torch.empty(x.shape, dtype=torch.int8, device=dev)
        scale = torch.empty(x.shape[0], dtype=torch.float32, device=dev)
        raise_for(flce_quantize_int8(DTYPES[_dtype_name(x)], _ptr(x), x.shape[0], x.shape[1], _ptr(q), _ptr(scale),
                                     stream_handle(dev)), "flce_quantize_int8")
    return q, scale


@by_pointers
def quantize_int8(x):
    """Rows of x (R, H) as 8-bit integers: (q int8 (R, H), scale fp32 (R,)), x ~ scale[:, None] * q, with
    scale = max|row| / 127.  For a weight (V, H) once, when a scorer is loaded.  H must be a multiple of 16.
    All-zero rows give scale 0, rows with NaN or infinities scale NaN.  Neither output has a gradient: x is a
    constant here, also where it requires one."""
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    _dtype_name(x)
    if x.shape[1] == 0 or x.shape[1] % 16:
        raise ValueError(f"rows must be a multiple of 16 long, got {x.shape[1]}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if x.device.type != "cuda":
        raise ValueError(f"x must be on a GPU, not {x.device}")
    return _quantize(x.detach())


def _check_int8(hidden, weight, weight_scale, targets, bias, hidden_scale):
    import torch
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError(f"hidden and weight must be 2-D, got {tuple(hidden.shape)} and {tuple(weight.shape)}")
    n, h = hidden.shape
    v = weight.shape[0]
    if weight.dtype != torch.int8:
        raise TypeError(f"weight must be int8 (quantize_int8), not {weight.dtype}")
    if hidden_scale is None:
        _dtype_name(hidden)
    elif hidden.dtype != torch.int8:
        raise TypeError(f"hidden must be int8 with hidden_scale, not {hidden.dtype}")
    if weight.shape[1] != h:
        raise ValueError(f"weight has {weight.shape[1]} columns, hidden has {h}")
    if h == 0 or h % 16:
        raise ValueError(f"hidden size must be a multiple of 16, got {h}")
    _targets_int32(targets)
    if targets.dim() != 1 or targets.shape[0] != n:
        raise ValueError(f"targets must have shape ({n},), got {tuple(targets.shape)}")
    vectors = [("weight_scale", weight_scale, v), ("bias", bias, v), ("hidden_scale", hidden_scale, n)]
    for name, t, size in vectors:
        if t is None:
            continue
        if t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32, not {t.dtype}")
        if t.dim() != 1 or t.shape[0] != size:
            raise ValueError(f"{name} must have shape ({size},), got {tuple(t.shape)}")
    named = [("hidden", hidden), ("weight", weight), ("targets", targets), *((k, t) for k, t, _ in vectors)]
    for name, t in named:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for name, t in named:
        if t is not None and (t.device.type != "cuda" or t.device != hidden.device):
            raise ValueError(f"{name} must be on hidden's GPU ({hidden.device}), not {t.device}")
    recorded = torch.is_grad_enabled()
    for name, t in named:
        if t is not None and ((recorded and t.requires_grad) or has_tangent(t)):
            raise ValueError(f"8-bit scores have no gradient: detach {name}, or use token_logprobs")


def _aligned16(t):
    """A vector as the kernels' entry point takes it: a slice of a vocabulary may begin anywhere (its rows of
    the weight are 16-byte aligned in any case)."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


@by_pointers
def token_logprobs_int8(hidden, weight, weight_scale, targets, bias=None, *, hidden_scale=None,
                        logit_scale: float = 1.0, softcap: Optional[float] = None, ignore_index: int = -100,
                        return_entropy: bool = False):
    """``token_logprobs`` of a frozen head held in 8 bits: weight int8 (V, H) and weight_scale fp32 (V,), from
    ``quantize_int8``.  hidden is fp32, bf16 or fp16 and is quantized here, token by token, or is int8 with its
    ``hidden_scale`` (N,).  The products are summed exactly, in int32.  bias (V,) is fp32.  No gradients."""
    import torch
    _check_int8(hidden, weight, weight_scale, targets, bias, hidden_scale)
    n, h = hidden.shape
    p = make_params(n, h, weight.shape[0], logit_scale=logit_scale, softcap=softcap, ignore_index=ignore_index,
                    reduction="none", targets_int32=_targets_int32(targets))
    dev = hidden.device
    with on_device(dev):
        ws_bytes = flce_logprobs_int8_workspace_size(p)
        weight_scale, bias = _aligned16(weight_scale), _aligned16(bias)
        if hidden_scale is None:
            hidden, hidden_scale = _quantize(hidden)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        logps, entropy, lse = (torch.empty(n, dtype=torch.float32, device=dev) for _ in range(3))
        raise_for(flce_logprobs_int8(p, _ptr(hidden), _ptr(hidden_scale), _ptr(weight), _ptr(weight_scale), _ptr(bias),
                                     _ptr(targets), _ptr(logps), _ptr(entropy), _ptr(lse), _ptr(workspace), ws_bytes,
                                     stream_handle(dev)), "flce_logprobs_int8")
    return (logps, entropy) if return_entropy else logps


# ----------------------------------------------------------------------------- 4-bit scoring

@functools.lru_cache(maxsize=None)
def _mx_ops():
    ops = torch_ops()
    return ops._quantize_mxfp4.default, ops._dequantize_mxfp4.default, ops._logprobs_mxfp4.default


@between_graphs
def quantize_mxfp4(x):
    """Rows of x (R, H) in MXFP4: (codes uint8 (R, H / 2), two to a byte, the earlier one in the low half; scales uint8
    (R, H / 32), byte s for 2^(s - 127)).  For a weight (V, H) once, when a scorer is loaded.  H must be a multiple of
    32, the values that share a scale.  A block with NaN or an infinity gives scale 255, which stands for NaN.
    Neither output has a gradient: x is a constant here, also where it requires one."""
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    _dtype_name(x)
    if x.shape[1] == 0 or x.shape[1] % 32:
        raise ValueError(f"rows must be a multiple of 32 long, got {x.shape[1]}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if not x.is_cuda:
        raise ValueError(f"x must be on a GPU, not {x.device}")
    return _mx_ops()[0](_aligned16(x))


def _check_mx(name, q, scale):
    import torch
    if q.dim() != 2 or scale.dim() != 2:
        raise ValueError(f"{name} and {name}_scale must be 2-D, got {tuple(q.shape)} and {tuple(scale.shape)}")
    if q.dtype != torch.uint8 or scale.dtype != torch.uint8:
        raise TypeError(f"{name} and {name}_scale must be uint8 (quantize_mxfp4), not {q.dtype} and {scale.dtype}")
    rows, cols = q.shape
    if cols == 0 or cols % 16:
        raise ValueError(f"rows of {name} must be a multiple of 16 bytes (32 values) long, got {cols}")
    if scale.shape != (rows, cols // 16):
        raise ValueError(f"{name}_scale must have shape {(rows, cols // 16)}, got {tuple(scale.shape)}")


@between_graphs
def dequantize_mxfp4(q, scale, dtype=None):
    """The values (R, H) that ``quantize_mxfp4``'s codes and scales stand for, in ``dtype`` (float32, the default,
    bfloat16 or float16; rounded where it does not hold them)."""
    import torch
    _check_mx("q", q, scale)
    dtype = torch.float32 if dtype is None else dtype
    if dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise TypeError(f"unsupported dtype {dtype}")
    for name, t in (("q", q), ("scale", scale)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for name, t in (("q", q), ("scale", scale)):
        if not t.is_cuda or t.device != q.device:
            raise ValueError(f"{name} must be on q's GPU ({q.device}), not {t.device}")
    return _mx_ops()[1](_aligned16(q), scale, dtype)


@functools.lru_cache(maxsize=1024)
def _mx_workspace(n, h, v, dtype, logit_scale, softcap, ignore_index, targets_int32):
    """Bytes of the call's workspace; refuses what the C entry point would."""
    return flce_logprobs_mxfp4_workspace_size(
        make_params(n, h, v, dtype=dtype, logit_scale=logit_scale, softcap=softcap, ignore_index=ignore_index,
                    reduction="none", targets_int32=targets_int32))


@between_graphs
def token_logprobs_mxfp4(hidden, weight, weight_scale, targets, bias=None, *, hidden_scale=None,
                         logit_scale: float = 1.0, softcap: Optional[float] = None, ignore_index: int = -100,
                         return_entropy: bool = False):
    """``token_logprobs`` of a frozen head held in MXFP4: weight uint8 (V, H / 2) and weight_scale uint8 (V, H / 32),
    from ``quantize_mxfp4``.  hidden (N, H) is fp32, bf16 or fp16 and is quantized here, or is uint8 codes (N, H / 2)
    with their ``hidden_scale`` (N, H / 32).  Products are exact and summed in fp32.  bias (V,) is fp32.  Vocabulary
    slices are taken (``weight[first:]``, ``weight_scale[first:]``).  No gradients."""
    import torch
    _check_mx("weight", weight, weight_scale)
    v, h = weight.shape[0], 2 * weight.shape[1]
    if hidden_scale is not None:
        _check_mx("hidden", hidden, hidden_scale)
        n, cols, dtype = hidden.shape[0], 2 * hidden.shape[1], "bf16"
    else:
        if hidden.dim() != 2:
            raise ValueError(f"hidden must be 2-D, got {tuple(hidden.shape)}")
        dtype = _dtype_name(hidden)
        n, cols = hidden.shape
    if cols != h:
        raise ValueError(f"weight has {h} columns, hidden has {cols}")
    int32 = _targets_int32(targets)
    if targets.dim() != 1 or targets.shape[0] != n:
        raise ValueError(f"targets must have shape ({n},), got {tuple(targets.shape)}")
    if bias is not None:
        if bias.dtype != torch.float32:
            raise TypeError(f"bias must be float32, not {bias.dtype}")
        if bias.dim() != 1 or bias.shape[0] != v:
            raise ValueError(f"bias must have shape ({v},), got {tuple(bias.shape)}")
    named = [("hidden", hidden), ("weight", weight), ("targets", targets), ("weight_scale", weight_scale)]
    if bias is not None:
        named.append(("bias", bias))
    if hidden_scale is not None:
        named.append(("hidden_scale", hidden_scale))
    dev = hidden.device
    for name, t in named:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not t.is_cuda or t.device != dev:
            raise ValueError(f"{name} must be on hidden's GPU ({dev}), not {t.device}")
    recorded = torch.is_grad_enabled()
    for name, t in (("hidden", hidden), ("bias", bias)):     # the others are integers
        if t is not None and ((recorded and t.requires_grad) or has_tangent(t)):
            raise ValueError(f"4-bit scores have no gradient: detach {name}, or use token_logprobs")
    logit_scale, softcap, ignore_index = float(logit_scale), float(softcap or 0.0), int(ignore_index)
    ws_bytes = _mx_workspace(n, h, v, dtype, logit_scale, softcap, ignore_index, int32)
    logps, entropy = _mx_ops()[2](_aligned16(hidden), _aligned16(hidden_scale), _aligned16(weight),
                                  _aligned16(weight_scale), _aligned16(bias), targets, logit_scale, softcap, ignore_index,
                                  ws_bytes, return_entropy)
    return (logps, entropy) if return_entropy else logps
