"""Token embedding: the torch side of flce_embedding_* (include/flce.h has the formulas).  The autograd node is C++
(csrc/flce_torch.cpp)."""
from __future__ import annotations

import functools
import math
from typing import Optional

from . import (DTYPES, FLCE_ACCUMULATE_GRAD_WEIGHT, FLCE_TARGETS_INT32, _dtype_name, _ptr, between_graphs, by_pointers,
               flce_embedding_backward, flce_embedding_params, flce_embedding_workspace_size, torch_ops)
from .logprobs import has_tangent, on_device, raise_for, stream_handle


@functools.lru_cache(maxsize=1024)
def _params(n, h, v, ignore_index, dtype, grad_dtype, flags, scale):
    return flce_embedding_params(n, h, v, ignore_index, dtype, grad_dtype, flags, scale)


@functools.lru_cache(maxsize=1024)
def _workspace(n, h, v):
    return flce_embedding_workspace_size(flce_embedding_params(n, h, v, -100, 0, 0, 0, 1.0))


def _check_ids(ids):
    import torch
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"ids must be int64 or int32, not {ids.dtype}")
    if ids.dim() != 1:
        raise ValueError(f"ids must be 1-D, got {tuple(ids.shape)}")
    return FLCE_TARGETS_INT32 if ids.dtype == torch.int32 else 0


def _check_places(named):
    for name, t in named:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    dev = named[0][1].device
    for name, t in named:
        if t is not None and (not t.is_cuda or t.device != dev):
            raise ValueError(f"{name} must be on {named[0][0]}' GPU ({dev}), not {t.device}")


def _check_scale(scale):
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")


def _run_backward(p, ids, grad, grad_weight):
    import torch
    dev = grad.device
    with on_device(dev):
        ws_bytes = _workspace(p.n_tokens, p.hidden, p.vocab)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        raise_for(flce_embedding_backward(p, _ptr(ids), _ptr(grad), _ptr(grad_weight), _ptr(workspace), ws_bytes,
                                          stream_handle(dev)), "flce_embedding_backward")
    return grad_weight


@functools.lru_cache(maxsize=None)
def _op():
    return torch_ops()._embedding.default


@between_graphs
def embedding(ids, weight, *, scale: float = 1.0, ignore_index: int = -100):
    """Rows ``scale * weight[ids]`` (N, H) in weight's dtype (fp32, bf16, fp16), differentiable in weight (V, H).

    ids (N,) are int64 or int32.  A token whose id is ``ignore_index``, or no row of weight, gives 0 and takes no
    gradient (so a slice of the vocabulary may be looked up with ``ids - first``).  The gradient is a whole (V, H)
    tensor; ``embedding_backward`` adds it to one that is there, as for a head that shares the weight."""
    _check_ids(ids)
    if weight.dim() != 2 or 0 in weight.shape:
        raise ValueError(f"weight must be 2-D and not empty, got {tuple(weight.shape)}")
    _dtype_name(weight)
    _check_scale(scale)
    _check_places([("ids", ids), ("weight", weight)])
    workspace = _workspace(ids.shape[0], weight.shape[1], weight.shape[0])
    if has_tangent(weight):
        raise NotImplementedError("embedding has no forward-mode derivative")
    return _op()(ids, weight, float(scale), int(ignore_index), workspace)


@by_pointers
def embedding_backward(grad, ids, vocab: int, *, scale: float = 1.0, ignore_index: int = -100,
                       grad_weight_dtype: Optional[str] = None, grad_weight=None):
    """The gradient (vocab, H) of ``embedding``'s weight from that of its output, grad (N, H), summed in fp32.

    If ``grad_weight`` is given, the gradient is added to it in place and the same tensor is returned: only the rows
    that occur are touched.  It is the way to train a tied head: pass the buffer of ``backward``'s grad_weight."""
    import torch
    flags = _check_ids(ids)
    if grad.dim() != 2 or grad.shape[0] != ids.shape[0] or grad.shape[1] < 1:
        raise ValueError(f"grad must have shape ({ids.shape[0]}, H), got {tuple(grad.shape)}")
    dtype = _dtype_name(grad)
    if vocab < 1:
        raise ValueError(f"vocab must be at least 1, got {vocab}")
    _check_scale(scale)
    if grad_weight is not None:
        grad_weight_dtype = _dtype_name(grad_weight)
        if tuple(grad_weight.shape) != (vocab, grad.shape[1]):
            raise ValueError(f"grad_weight must have shape {(vocab, grad.shape[1])}, got {tuple(grad_weight.shape)}")
        flags |= FLCE_ACCUMULATE_GRAD_WEIGHT
    elif grad_weight_dtype is not None and grad_weight_dtype not in DTYPES:
        raise ValueError(f"invalid grad_weight_dtype {grad_weight_dtype!r}")
    _check_places([("ids", ids), ("grad", grad), ("grad_weight", grad_weight)])
    grad_weight_dtype = grad_weight_dtype or dtype
    p = _params(ids.shape[0], grad.shape[1], int(vocab), int(ignore_index), DTYPES[dtype], DTYPES[grad_weight_dtype], flags,
                float(scale))
    if grad_weight is None:
        kinds = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
        grad_weight = torch.empty((vocab, grad.shape[1]), dtype=kinds[grad_weight_dtype], device=grad.device)
    return _run_backward(p, ids, grad, grad_weight)
