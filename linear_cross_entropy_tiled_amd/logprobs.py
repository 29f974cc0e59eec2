"""Per-token log-probabilities and entropies of a linear head: the torch side of
flce_logprobs_* (include/flce.h has the formulas)."""
from __future__ import annotations

import contextlib
import functools
from typing import Optional

from . import (FLCE_OK, FLCE_PASS_BACKWARD, FLCE_PASS_FORWARD, FlceError, _ptr, _stream_handle, _targets_int32,
               _validate, flce_logprobs_backward, flce_logprobs_forward, flce_logprobs_workspace_size, make_params)


def on_device(device):
    """The library launches on the current device: makes it the tensors'."""
    import torch
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


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
                                        _ptr(entropy), _ptr(lse), _ptr(workspace), ws_bytes, _stream_handle(dev)),
                  "flce_logprobs_forward")
    return logps, entropy, lse


def _upstream(g):
    import torch
    return None if g is None else g.to(torch.float32).contiguous()


@functools.lru_cache(maxsize=None)
def _function():
    import torch
    from torch.autograd.function import once_differentiable

    class TokenLogprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, hidden, weight, bias, targets, p):
            logps, entropy, lse = _forward(p, hidden, weight, bias, targets)
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(hidden, weight, bias, targets, lse, entropy)
            ctx.p = p
            return logps, entropy

        @staticmethod
        @once_differentiable
        def backward(ctx, g, h):
            if g is None and h is None:
                return (None,) * 5
            hidden, weight, bias, targets, lse, entropy = ctx.saved_tensors
            g, h = _upstream(g), _upstream(h)
            dev = hidden.device
            with on_device(dev):
                ws_bytes = flce_logprobs_workspace_size(ctx.p, FLCE_PASS_BACKWARD)
                workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
                gh, gw = torch.empty_like(hidden), torch.empty_like(weight)
                gb = None if bias is None else torch.empty_like(bias)
                raise_for(flce_logprobs_backward(ctx.p, _ptr(hidden), _ptr(weight), _ptr(bias), _ptr(targets),
                                                 _ptr(lse), _ptr(entropy), _ptr(g), _ptr(h), _ptr(gh), _ptr(gw),
                                                 _ptr(gb), _ptr(workspace), ws_bytes, _stream_handle(dev)),
                          "flce_logprobs_backward")
            return gh, gw, gb, None, None

    return TokenLogprobs


def token_logprobs(hidden, weight, targets, bias=None, *, logit_scale: float = 1.0, softcap: Optional[float] = None,
                   ignore_index: int = -100, return_entropy: bool = False, vocab_chunk: int = 0):
    """Log-probabilities (N,) of ``targets`` under softmax(softcap(logit_scale (hidden @ weight.T + bias))),
    in fp32, without the (N, V) logits; with ``return_entropy`` also each row's entropy (nats).

    Both are differentiable in hidden, weight and bias (the backward recomputes the logit tiles).
    Rows whose target is ``ignore_index`` give 0 and take no gradient.  ``vocab_chunk``: as in
    ``backward``.  hidden, weight and bias share one dtype (fp32, bf16, fp16)."""
    dt = _validate(hidden, weight, targets, bias, reduction="none")
    p = make_params(hidden.shape[0], hidden.shape[1], weight.shape[0], dtype=dt, logit_scale=logit_scale,
                    softcap=softcap, ignore_index=ignore_index, reduction="none",
                    targets_int32=_targets_int32(targets), vocab_chunk=vocab_chunk)
    logps, entropy = _function().apply(hidden, weight, bias, targets, p)
    return (logps, entropy) if return_entropy else logps
