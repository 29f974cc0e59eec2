"""fp64 oracle of the alignment operators, from their definitions: per-token
log-probabilities and entropies of a linear head with their gradients, the
paired preference loss and the clipped policy loss.  Independent of the library;
sequence by sequence and row by row, in plain numpy."""
from __future__ import annotations

import numpy as np


# ----------------------------------------------------------------------------- log-probabilities

def token_logprobs(hidden, weight, bias, targets, *, logit_scale=1.0, softcap=0.0, ignore_index=-100,
                   product=None):
    """(logp, entropy, z, dz/du) per row; ignored and out-of-range rows are 0.  ``product``: the
    rows' hidden . weight^T, where it is not that of hidden and weight."""
    u = (hidden @ weight.T if product is None else product)
    if bias is not None:
        u = u + bias
    u = logit_scale * u
    slope = np.ones_like(u)
    z = u
    if softcap:
        t = np.tanh(u / softcap)
        z, slope = softcap * t, 1.0 - t * t
    n, v = z.shape
    valid = (targets != ignore_index) & (targets >= 0) & (targets < v)
    logp, entropy = np.zeros(n), np.zeros(n)
    for i in np.flatnonzero(valid):
        m = z[i].max()
        with np.errstate(invalid="ignore", divide="ignore"):
            e = np.exp(z[i] - m)
            lse = m + np.log(e.sum())
            lp = z[i] - lse
            p = np.exp(lp)
            logp[i] = lp[targets[i]]
            entropy[i] = -np.sum(np.where(p > 0, p * lp, 0.0 * p))
    return logp, entropy, z, slope * logit_scale


def token_logprobs_grads(hidden, weight, bias, targets, grad_logp, grad_entropy, **opts):
    logp, entropy, z, slope = token_logprobs(hidden, weight, bias, targets, **opts)
    n, v = z.shape
    valid = (targets != opts.get("ignore_index", -100)) & (targets >= 0) & (targets < v)
    d = np.zeros_like(z)
    for i in np.flatnonzero(valid):
        m = z[i].max()
        lse = m + np.log(np.exp(z[i] - m).sum())
        lp = z[i] - lse
        p = np.exp(lp)
        d[i] = -grad_logp[i] * p - grad_entropy[i] * np.where(p > 0, p * (lp + entropy[i]), 0.0)
        d[i, targets[i]] += grad_logp[i]
    d *= slope
    return d @ weight, d.T @ hidden, d.sum(0)


def quantize_int8(x):
    """Rows as 8-bit integers and fp32 scales; the definition is in fp32 operations:
    s = max|x| * fp32(1/127), q = rint(x * fp32(1/s)), rows below 1e-30 and rows that are
    not finite have q = 0."""
    x = np.asarray(x, dtype=np.float32)
    top = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    s = (top * np.float32(1.0 / 127.0)).astype(np.float32)
    ok = np.isfinite(top) & (top >= np.float32(1e-30))
    r = np.where(ok, np.float32(1.0) / np.where(ok, s, np.float32(1.0)), np.float32(0.0)).astype(np.float32)
    q = np.clip(np.rint(np.where(ok[:, None], x, np.float32(0.0)) * r[:, None]), -127, 127).astype(np.int8)
    s = np.where(np.isfinite(top), np.where(ok, s, np.float32(0.0)), np.float32(np.nan)).astype(np.float32)
    return q, s


# ----------------------------------------------------------------------------- sequences

def sequences(shape, offsets, mask):
    """The flat indices of each sequence's kept tokens."""
    if offsets is None:
        s, length = shape
        spans = [(i * length, (i + 1) * length) for i in range(s)]
    else:
        spans = list(zip(offsets[:-1], offsets[1:]))
    flat = np.ones(int(np.prod(shape)), dtype=bool) if mask is None else np.asarray(mask).reshape(-1) != 0
    return [np.arange(b, e)[flat[b:e]] for b, e in spans]


def preference(logps, ref, offsets=None, mask=None, *, beta=0.1, loss_type="sigmoid", label_smoothing=0.0,
               margin=0.0, length_normalize=False, reduction="mean"):
    """(loss per pair or reduced, rewards, d(sum of g loss)/d logps as a function of g)."""
    seqs = sequences(logps.shape, offsets, mask)
    x = logps.reshape(-1) - (0.0 if ref is None else ref.reshape(-1))
    pairs = len(seqs) // 2
    per = np.array([1.0 / max(len(s), 1) if length_normalize else 1.0 for s in seqs])
    rewards = np.array([beta * np.sum(x[s]) for s in seqs]) * per if seqs else np.zeros(0)
    h = rewards[:pairs] - rewards[pairs:] - margin
    if loss_type == "sigmoid":
        soft = np.logaddexp(0.0, -h)
        loss = (1 - label_smoothing) * soft + label_smoothing * np.logaddexp(0.0, h)
        slope = -(1 - label_smoothing) * np.exp(-np.logaddexp(0.0, h)) + label_smoothing * np.exp(-soft)
    elif loss_type == "hinge":
        loss, slope = np.maximum(0.0, 1 - h), np.where(h < 1, -1.0, 0.0)
    else:
        loss, slope = (h / beta - 0.5 / beta) ** 2, 2 * (h / beta - 0.5 / beta) / beta
    share = 1.0 / max(pairs, 1) if reduction == "mean" else 1.0

    def grad(g):
        g = np.broadcast_to(np.asarray(g, dtype=np.float64), (pairs,)) * share
        out = np.zeros(x.shape)
        for k, s in enumerate(seqs):
            p = k % pairs
            out[s] = (1.0 if k < pairs else -1.0) * g[p] * slope[p] * beta * per[k]
        return out.reshape(logps.shape)

    if reduction == "mean":
        loss = loss.mean() if pairs else np.nan
    elif reduction == "sum":
        loss = loss.sum()
    return loss, rewards, grad


def policy(logps, old, advantages, ref=None, entropy=None, offsets=None, mask=None, *, clip_low=0.2, clip_high=0.2,
           dual_clip=None, kl_coef=0.0, entropy_coef=0.0, reduction="mean"):
    """dict(loss, grad(g), grad_entropy(g), terms: sum of the absolute terms per token, metrics)."""
    seqs = sequences(logps.shape, offsets, mask)
    lp, old = logps.reshape(-1), old.reshape(-1)
    t = lp.size
    adv = np.zeros(t)
    if advantages.size == t and advantages.shape == logps.shape:
        adv[:] = advantages.reshape(-1)
    else:
        for k, s in enumerate(seqs):
            adv[s] = advantages.reshape(-1)[k]
    kept = np.zeros(t, dtype=bool)
    weight = np.zeros(t)
    filled = sum(len(s) > 0 for s in seqs)
    total = sum(len(s) for s in seqs)
    for s in seqs:
        kept[s] = True
        if len(s):
            weight[s] = {"mean": 1.0 / total, "sequence_mean": 1.0 / (len(s) * filled)}.get(reduction, 1.0)
    loss, d, size, k, cut = np.zeros(t), np.zeros(t), np.zeros(t), np.zeros(t), np.zeros(t, dtype=bool)
    i = np.flatnonzero(kept)
    r, a = np.exp(lp[i] - old[i]), adv[i]
    lo, hi = 1 - clip_low, 1 + clip_high
    plain = np.where(a == 0, 0.0, r * a)
    bound = np.clip(r, lo, hi) * a
    active = (plain <= bound) | np.isnan(plain)
    gain = np.where(active, plain, bound)
    if dual_clip is not None:
        far = (a < 0) & (r > dual_clip)
        gain, active = np.where(far, dual_clip * a, gain), active & ~far
    loss[i], d[i], size[i], cut[i] = -gain, np.where(active, -plain, 0.0), np.abs(gain) + np.abs(plain), ~active
    if ref is not None:
        away = ref.reshape(-1)[i] - lp[i]
        k[i] = np.expm1(away) - away
        loss[i] += kl_coef * k[i]
        d[i] -= kl_coef * np.expm1(away)
        size[i] += np.abs(kl_coef) * (np.abs(k[i]) + np.abs(np.expm1(away)) + np.abs(away))
    if entropy is not None:
        loss[i] -= entropy_coef * entropy.reshape(-1)[i]
        size[i] += np.abs(entropy_coef * entropy.reshape(-1)[i])
    if reduction == "none":
        value = loss.reshape(logps.shape)
    elif total == 0:
        value = 0.0 if reduction == "sum" else np.nan
    else:
        value = float(np.sum(loss[i] * weight[i]))

    def spread(g, x):
        g = np.broadcast_to(np.asarray(g, dtype=np.float64), logps.shape).reshape(-1)
        out = np.zeros(t)
        out[i] = g[i] * weight[i] * x[i]
        return out.reshape(logps.shape)

    return dict(loss=value, grad=lambda g: spread(g, d), grad_entropy=lambda g: spread(g, np.full(t, -entropy_coef)),
                terms=(size * weight).reshape(logps.shape), num_tokens=total,
                clip_fraction=cut.sum() / total if total else np.nan, kl=k.sum() / total if total else np.nan)
