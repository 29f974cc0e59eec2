"""Preference and policy losses over per-token log-probabilities: the torch side
of flce_preference_* and flce_policy_* (include/flce.h has the formulas).

Token tensors are (S, L), with any row stride and contiguous rows, or, with
``offsets`` (S + 1 int64 or int32 values on the GPU), one packed (T,) tensor in
which sequence s is ``[offsets[s], offsets[s + 1])``.  ``mask`` (bool or uint8,
the tokens' shape) says which tokens count; nothing that a masked token holds is
used, NaN and infinities included, and its gradient is 0.

Everything runs on the current stream; nothing synchronises.
"""
from __future__ import annotations

import functools
import math
from typing import Optional

from . import (DTYPES, REDUCTIONS, _dtype_name, _ptr, by_pointers, flce_policy_backward,
               flce_policy_forward, flce_policy_params, flce_policy_workspace_size, flce_preference_backward,
               flce_preference_forward, flce_preference_params, flce_preference_workspace_size, flce_token_view)
from .logprobs import differentiable, first_order, on_device, raise_for, stream_handle, upstream

PREFERENCE_TYPES = {"sigmoid": 0, "hinge": 1, "squared": 2}
POLICY_REDUCTIONS = {**REDUCTIONS, "sequence_mean": 3}
FLCE_OFFSETS_INT32 = 1
FLCE_ADVANTAGE_PER_SEQUENCE = 2


def _check_rows(t, name):
    """Rows are read as contiguous; only the distance between them is free."""
    if t.dim() == 1:
        ok = t.stride(0) == 1 or t.shape[0] <= 1
    else:
        ok = (t.stride(1) == 1 or t.shape[1] <= 1) and (t.stride(0) >= t.shape[1] or t.shape[0] <= 1)
    if not ok and t.numel() > 0:
        raise ValueError(f"{name} must have contiguous rows that do not overlap, got strides {t.stride()}")


def _view(t):
    if t is None:
        return flce_token_view(None, 0)
    return flce_token_view(t.data_ptr(), t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else 0)


def _check_tokens(logps, others, offsets, mask, constants, per_sequence=()):
    """Types, shapes, layout and device of the token tensors.  The kernels trust all of them.
    Returns (n_seqs, length, flags)."""
    import torch
    dtype, shape, dev = logps.dtype, logps.shape, logps.device
    _dtype_name(logps)
    named = [("logps", logps), *((name, t) for name, t in others if t is not None)]
    for name, t in named:
        if t.dtype != dtype:
            raise TypeError(f"{name} dtype {t.dtype} differs from logps' {dtype}")
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"mask must be bool or uint8, not {mask.dtype}")
        named.append(("mask", mask))
    flags = 0
    if offsets is None:
        if len(shape) != 2:
            raise ValueError(f"logps must be (S, L), or (T,) with offsets, got {tuple(shape)}")
        n_seqs, length = shape
    else:
        if offsets.dtype not in (torch.int64, torch.int32):
            raise TypeError(f"offsets must be int64 or int32, not {offsets.dtype}")
        if offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError(f"offsets must hold S + 1 values, got shape {tuple(offsets.shape)}")
        if len(shape) != 1:
            raise ValueError(f"packed logps must be (T,), got {tuple(shape)}")
        n_seqs, length = offsets.shape[0] - 1, shape[0]
        flags = FLCE_OFFSETS_INT32 if offsets.dtype == torch.int32 else 0
        if not offsets.is_contiguous():
            raise ValueError("offsets must be contiguous")
    for name, t in named:
        if t.shape != shape:
            raise ValueError(f"{name} must have logps' shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            _check_rows(t, name)
    for name, t in (*named, ("offsets", offsets), *per_sequence):
        if t is not None and (t.device != dev or not t.is_cuda):
            raise ValueError(f"{name} must be on logps' GPU ({dev}), not {t.device}")
    if torch.is_grad_enabled():
        for name, t in constants:
            if t is not None and t.requires_grad:
                raise ValueError(f"{name} is a constant of the loss and gets no gradient: detach it")
    return n_seqs, length, flags


@functools.lru_cache(maxsize=1024)
def _preference_workspace(n_seqs, length):
    return flce_preference_workspace_size(flce_preference_params(n_seqs, length, beta=1.0))


@functools.lru_cache(maxsize=1024)
def _policy_workspace(n_seqs, length):
    return flce_policy_workspace_size(flce_policy_params(n_seqs, length))


# ----------------------------------------------------------------------------- preference loss

def _preference_forward(p, logps, ref, mask, offsets):
    import torch
    dev = logps.device
    pairs = p.n_seqs // 2
    with on_device(dev):
        ws_bytes = _preference_workspace(p.n_seqs, p.length)
        # one allocation: the workspace, then the sequences' gradient factors for the backward
        kept = torch.empty(ws_bytes // 4 + p.n_seqs, dtype=torch.float32, device=dev)
        loss = torch.empty((pairs,) if p.reduction == 0 else (), dtype=torch.float32, device=dev)
        rewards = torch.empty(p.n_seqs, dtype=torch.float32, device=dev)
        raise_for(flce_preference_forward(p, _view(logps), _view(ref), _view(mask), _ptr(offsets), _ptr(loss),
                                          _ptr(rewards), kept.data_ptr() + ws_bytes, _ptr(kept), ws_bytes,
                                          stream_handle(dev)), "flce_preference_forward")
    return loss, rewards, kept


@functools.lru_cache(maxsize=None)
def _preference_function():
    import torch

    class PreferenceLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logps, ref, mask, offsets, p):
            loss, rewards, kept = _preference_forward(p, logps, ref, mask, offsets)
            ctx.mark_non_differentiable(rewards)
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(kept, mask, offsets)
            ctx.p, ctx.like = p, (logps.shape, logps.dtype, logps.device)
            return loss, rewards

        @first_order
        def backward(ctx, g, _):
            if g is None:
                return (None,) * 5
            kept, mask, offsets = ctx.saved_tensors
            shape, dtype, dev = ctx.like
            g = upstream(g)
            grad = torch.empty(shape, dtype=dtype, device=dev)
            with on_device(dev):
                raise_for(flce_preference_backward(ctx.p, _ptr(g), kept.data_ptr() + 4 * (kept.numel() - ctx.p.n_seqs),
                                                   _view(mask), _ptr(offsets),
                                                   _ptr(grad), stream_handle(dev)), "flce_preference_backward")
            return grad, None, None, None, None

    return PreferenceLoss


@by_pointers
def preference_loss(logps, ref_logps=None, *, offsets=None, mask=None, beta: float = 0.1, loss_type: str = "sigmoid",
                    label_smoothing: float = 0.0, margin: float = 0.0, length_normalize: bool = False,
                    reduction: str = "mean", return_metrics: bool = False):
    """Paired preference loss from per-token log-probabilities, differentiable in ``logps``.

    The first half of the sequences are the chosen answers, the second half the rejected ones of
    the same pairs.  R_s sums logps - ref_logps (or logps, without a reference) over a sequence's
    kept tokens, divided by their number with ``length_normalize``; h = beta (R_chosen -
    R_rejected) - margin; the loss of a pair is
      "sigmoid"  -(1 - label_smoothing) log sigmoid(h) - label_smoothing log sigmoid(-h)
      "hinge"    max(0, 1 - h)
      "squared"  (h / beta - 1 / (2 beta))^2.
    Returns the fp32 loss (one value, or one per pair for "none"); with ``return_metrics`` also
    {"chosen_rewards", "rejected_rewards"}: beta R of each pair's answers."""
    if reduction not in REDUCTIONS:
        raise ValueError(f"invalid reduction {reduction!r}")
    if loss_type not in PREFERENCE_TYPES:
        raise ValueError(f"invalid loss_type {loss_type!r}")
    if not (math.isfinite(beta) and beta > 0):
        raise ValueError(f"beta must be positive, got {beta}")
    if not 0 <= label_smoothing <= 1 or (label_smoothing and loss_type != "sigmoid"):
        raise ValueError(f"label_smoothing must be within [0, 1], and 0 unless loss_type is 'sigmoid', "
                         f"got {label_smoothing}")
    if not math.isfinite(margin):
        raise ValueError(f"margin must be finite, got {margin}")
    n_seqs, length, flags = _check_tokens(logps, [("ref_logps", ref_logps)], offsets, mask,
                                          [("ref_logps", ref_logps)])
    if n_seqs % 2:
        raise ValueError(f"an even number of sequences is needed (chosen, then rejected), got {n_seqs}")
    p = flce_preference_params(n_seqs, length, DTYPES[_dtype_name(logps)], REDUCTIONS[reduction],
                               PREFERENCE_TYPES[loss_type], flags, 1 if length_normalize else 0, 0, beta,
                               label_smoothing, margin)
    if differentiable(logps, ref_logps):
        loss, rewards = _preference_function().apply(logps, ref_logps, mask, offsets, p)
    else:
        loss, rewards, _ = _preference_forward(p, logps, ref_logps, mask, offsets)
    if not return_metrics:
        return loss
    return loss, {"chosen_rewards": rewards[:n_seqs // 2], "rejected_rewards": rewards[n_seqs // 2:]}


# ----------------------------------------------------------------------------- policy loss

def _policy_forward(p, logps, old, ref, entropy, advantages, mask, offsets, needs_grad, metrics):
    import torch
    dev = logps.device
    with on_device(dev):
        ws_bytes = _policy_workspace(p.n_seqs, p.length)
        # one allocation: the workspace, then for the backward the tokens' gradients (16-byte
        # aligned) and the weights
        n_unit = (logps.numel() + 3) // 4 * 4 if needs_grad else 0
        kept = torch.empty(ws_bytes // 4 + n_unit + 1 + p.n_seqs, dtype=torch.float32, device=dev)
        at = kept.data_ptr()
        loss = torch.empty(logps.shape if p.reduction == 0 else (), dtype=torch.float32, device=dev)
        per_seq = p.flags & FLCE_ADVANTAGE_PER_SEQUENCE
        adv = flce_token_view(advantages.data_ptr(), 0) if per_seq else _view(advantages)
        raise_for(flce_policy_forward(p, _view(logps), _view(old), _view(ref), _view(entropy), adv, _view(mask),
                                       _ptr(offsets), _ptr(loss), at + ws_bytes if n_unit else None,
                                      at + ws_bytes + 4 * n_unit, _ptr(metrics), at, ws_bytes, stream_handle(dev)),
                  "flce_policy_forward")
    return loss, kept, ws_bytes, n_unit


@functools.lru_cache(maxsize=None)
def _policy_function():
    import torch

    class PolicyLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logps, entropy, old, ref, advantages, mask, offsets, p, metrics):
            loss, kept, ctx.unit_at, ctx.n_unit = _policy_forward(p, logps, old, ref, entropy, advantages, mask,
                                                                  offsets, ctx.needs_input_grad[0], metrics)
            ctx.save_for_backward(kept, mask, offsets)
            ctx.p, ctx.like = p, (logps.shape, logps.dtype, logps.device)
            return loss

        @first_order
        def backward(ctx, g):
            kept, mask, offsets = ctx.saved_tensors
            unit = kept.data_ptr() + ctx.unit_at
            shape, dtype, dev = ctx.like
            g = upstream(g)
            grads = [torch.empty(shape, dtype=dtype, device=dev) if need else None
                     for need in ctx.needs_input_grad[:2]]
            with on_device(dev):
                raise_for(flce_policy_backward(ctx.p, _ptr(g), unit if ctx.n_unit else None,
                                               unit + 4 * ctx.n_unit, _view(mask), _ptr(offsets), _ptr(grads[0]),
                                               _ptr(grads[1]), stream_handle(dev)), "flce_policy_backward")
            return (*grads, None, None, None, None, None, None, None)

    return PolicyLoss


@by_pointers
def policy_loss(logps, old_logps, advantages, *, ref_logps=None, entropy=None, offsets=None, mask=None,
                clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: Optional[float] = None,
                kl_coef: float = 0.0, entropy_coef: float = 0.0, reduction: str = "mean",
                return_metrics: bool = False, advantages_per_sequence: Optional[bool] = None):
    """Clipped policy loss with a KL term, differentiable in ``logps`` and ``entropy``.

    Per kept token, with r = exp(logps - old_logps) and A its advantage:
      s = min(r A, clip(r, 1 - clip_low, 1 + clip_high) A); for A < 0 and ``dual_clip`` c: max(s, c A)
      k = e^d - d - 1 with d = ref_logps - logps
      loss = -s + kl_coef k - entropy_coef entropy,  a term with coefficient 0 left out
    ``advantages`` (fp32): the tokens' shape, or one value per sequence, (S,) or (S, 1).  A packed batch
    with as many tokens as sequences leaves (S,) open: ``advantages_per_sequence`` says which.
    ``reduction``: "mean" over the kept tokens, "sequence_mean" (mean over sequences of each one's
    mean, sequences without a kept token left out), "sum", or "none" (the tokens' shape).  A mean of
    nothing is NaN, with zero gradients.
    Returns the fp32 loss; with ``return_metrics`` also {"num_tokens" (int64), "clip_fraction",
    "kl"}: tokens kept, the share whose gradient a clip cuts off, and the mean of k."""
    import torch
    if reduction not in POLICY_REDUCTIONS:
        raise ValueError(f"invalid reduction {reduction!r}")
    if not (clip_low >= 0 and clip_high >= 0):
        raise ValueError(f"clip_low and clip_high must be at least 0, got {clip_low} and {clip_high}")
    if dual_clip is not None and not (math.isfinite(dual_clip) and dual_clip > 1):
        raise ValueError(f"dual_clip must be above 1, got {dual_clip}")
    if not (math.isfinite(kl_coef) and math.isfinite(entropy_coef)):
        raise ValueError(f"kl_coef and entropy_coef must be finite, got {kl_coef} and {entropy_coef}")
    if kl_coef and ref_logps is None:
        raise ValueError("kl_coef needs ref_logps")
    if entropy_coef and entropy is None:
        raise ValueError("entropy_coef needs entropy")
    if advantages.dtype != torch.float32:
        raise TypeError(f"advantages must be float32, not {advantages.dtype}")
    others = [("old_logps", old_logps), ("ref_logps", ref_logps), ("entropy", entropy)]
    constants = [("old_logps", old_logps), ("ref_logps", ref_logps), ("advantages", advantages)]
    n_seqs, length, flags = _check_tokens(logps, others, offsets, mask, constants, [("advantages", advantages)])
    per_token = advantages.shape == logps.shape
    per_seq = tuple(advantages.shape) in ((n_seqs,), (n_seqs, 1))
    if advantages_per_sequence is not None:
        per_token, per_seq = per_token and not advantages_per_sequence, per_seq and advantages_per_sequence
    if not (per_token or per_seq):
        wanted = {None: f"logps' shape {tuple(logps.shape)} or ({n_seqs},)", True: f"shape ({n_seqs},)",
                  False: f"logps' shape {tuple(logps.shape)}"}[advantages_per_sequence]
        raise ValueError(f"advantages must have {wanted}, got {tuple(advantages.shape)}")
    if per_token and per_seq and advantages.dim() == 1 and n_seqs > 1:
        raise ValueError(f"advantages of shape {tuple(advantages.shape)} could be per token or per sequence: "
                         "say advantages_per_sequence=True or False")
    per_seq = not per_token
    if per_seq:
        if n_seqs > 1 and advantages.stride(0) != 1:
            raise ValueError("advantages must be contiguous")
        flags |= FLCE_ADVANTAGE_PER_SEQUENCE
    else:
        _check_rows(advantages, "advantages")
    p = flce_policy_params(n_seqs, length, DTYPES[_dtype_name(logps)], POLICY_REDUCTIONS[reduction], flags, 0,
                           clip_low, clip_high, dual_clip or 0.0, kl_coef, entropy_coef)
    metrics = torch.empty(2, dtype=torch.int64, device=logps.device) if return_metrics else None
    if differentiable(logps, entropy, old_logps, ref_logps, advantages):
        loss = _policy_function().apply(logps, entropy, old_logps, ref_logps, advantages, mask, offsets, p, metrics)
    else:
        loss, *_ = _policy_forward(p, logps, old_logps, ref_logps, entropy, advantages, mask, offsets, False, metrics)
    if not return_metrics:
        return loss
    both = metrics.view(torch.float32)
    return loss, {"num_tokens": metrics[0], "clip_fraction": both[2], "kl": both[3]}
