"""A softcap's own error is relative to the logit, not to the cap, in every kernel and type.

Tolerances, before any run: w = v / cap (two roundings), tanh(w) within 4 x 2^-24 of itself (a polynomial's last
operations up to 0.8; beyond, where tanh > 0.66, 1 - 2 r with r < 0.17 off by 3 x 2^-24 of itself), times the cap (one):
8 x 2^-24 |z|, besides what test_gpu_token_logprobs.py and test_gpu_logprobs_int8.py derive without a cap."""
import numpy as np
import pytest

from oracle import alignment_oracle as ao
from test_gpu_logprobs_int8 import _problem
from test_gpu_token_logprobs import U32, _bounds, _np, _tensors

pytestmark = pytest.mark.gpu
# 1000 tokens: large tiles; 100: small ones in most types; 16: the narrow ones
SHAPES = [(16, 64, 2000), (100, 64, 2000), (1000, 64, 16001)]


def _rows(n):
    """All rows, or some of each token tile."""
    return np.arange(n) if n <= 100 else np.unique(np.r_[0:8, 250:262, 508:516, n - 8:n])


def _check(lp, ent, z, t, ez, own):
    """Values of some rows against their fp64 logits z."""
    m = z.max(axis=1, keepdims=True)
    lse = m + np.log(np.exp(z - m).sum(axis=1, keepdims=True))
    l = z - lse
    valid = t >= 0
    want_h = -(np.exp(l) * l).sum(axis=1)
    at = np.maximum(t, 0)
    ez = ez + 8 * U32 * np.abs(z).max(axis=1)
    own = own * U32 * (np.abs(z).max(axis=1) + np.log(z.shape[1]) + 1)
    spread = 1 + 2 * (z.max(axis=1) - z.min(axis=1) + np.log(z.shape[1]))
    off = np.abs(lp - l[np.arange(len(t)), at]) / (2 * ez + own)
    off_h = np.abs(ent - want_h) / (spread * ez + 2 * own)
    assert off[valid].max() <= 1 and off_h[valid].max() <= 1, (off[valid].max(), off_h[valid].max())


@pytest.mark.parametrize("cap", [30.0, 1e3, 1e5])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_values(flce_lib, n, h, v, dtype, bias, cap):
    x, w, b, t = _tensors(n, h, v, dtype, seed=n + 1, bias=bias)
    lp, ent = flce_lib.token_logprobs(x.cuda(), w.cuda(), t.cuda(), b.cuda() if bias else None, softcap=cap,
                                      logit_scale=1.5, return_entropy=True)
    r = _rows(n)
    X, W, B = _np(x)[r], _np(w), _np(b)
    u = 1.5 * (X @ W.T + (0 if B is None else B))
    _check(_np(lp)[r], _np(ent)[r], cap * np.tanh(u / cap), t.numpy()[r],
           _bounds(X, W, B, dtype, dict(logit_scale=1.5)), 8)


@pytest.mark.parametrize("cap", [30.0, 1e3, 1e5])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("n,h,v", SHAPES)
def test_int8_values(flce_lib, n, h, v, bias, cap):
    x, w, b, t = _problem(n, h, v, seed=n + 2, bias=bias)
    wq, ws = flce_lib.quantize_int8(w.cuda())
    lp, ent = flce_lib.token_logprobs_int8(x.cuda(), wq, ws, t.cuda(), b.cuda() if bias else None, softcap=cap,
                                           logit_scale=1.5, return_entropy=True)
    r = _rows(n)
    q, s = ao.quantize_int8(x.float().numpy()[r])
    product = (q.astype(np.float64) @ wq.cpu().numpy().astype(np.float64).T) * s.astype(np.float64)[:, None] * _np(ws)[None]
    B = 0 if b is None else _np(b)
    u = 1.5 * (product + B)
    ez = 5 * U32 * 1.5 * (np.abs(product).max(axis=1) + np.abs(B).max())
    _check(_np(lp)[r], _np(ent)[r], cap * np.tanh(u / cap), t.numpy()[r], ez, 24)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("which", ["both", "entropy"])
def test_gradients_at_a_large_cap(flce_lib, n, h, v, dtype, bias, which):
    """The gradients of a cap that no logit comes near are those without a cap, in every row of hidden and
    weight: p is off by the logits' error and the logit gradient by its type's rounding, both times."""
    import torch
    x, w, b, t = _tensors(n, h, v, dtype, seed=n + 3, bias=bias)
    leaves = [a.cuda().requires_grad_(True) for a in (x, w, b) if a is not None]
    gen = torch.Generator().manual_seed(1)
    g, e = (torch.randn(n, generator=gen).cuda() for _ in range(2))
    if which == "entropy":      # every term is a p's
        g.zero_()

    def grads(**cap):
        lp, ent = flce_lib.token_logprobs(leaves[0], leaves[1], t.cuda(), leaves[2] if bias else None,
                                          return_entropy=True, **cap)
        return torch.autograd.grad((lp, ent), leaves, (g, e))

    got, plain = grads(softcap=1e5), grads()
    X, W, B, T = _np(x), _np(w), _np(b), t.numpy()
    logp, ent64, z, _ = ao.token_logprobs(X, W, B, T)
    # z = cap tanh(z / cap) differs from z by |z|^3 / (3 cap^2), the slope from 1 by (z / cap)^2: below 1e-8 here
    assert np.abs(z).max() < 8
    lse = z.max(axis=1) + np.log(np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1))
    l = z - lse[:, None]
    valid = T >= 0
    p = np.exp(l) * valid[:, None]
    G, Eg = np.abs(_np(g))[:, None], np.abs(_np(e))[:, None]
    a = G * p + Eg * p * (np.abs(l) + ent64[:, None])
    a[np.arange(n)[valid], T[valid]] += G[valid, 0]
    ez = (_bounds(X, W, B, dtype, {}) + 8 * U32 * np.abs(z).max(axis=1))[:, None]
    half = {"f16": 2.0 ** -11, "f32": 2.0 ** -24}[dtype]
    tiny = 2.0 ** -24 if dtype == "f16" else 0.0
    d_err = 2 * (a * (half + (4 + 2 * np.abs(l)) * (ez + 16 * U32 * (1 + np.abs(z) + np.abs(l))) + 8 * U32)
                 + tiny * a.max())
    for k, (err, size) in enumerate(((d_err @ np.abs(W), a @ np.abs(W)), (d_err.T @ np.abs(X), a.T @ np.abs(X)),
                                     (d_err.sum(0), a.sum(0)))[:len(leaves)]):
        one, two = _np(got[k]), _np(plain[k])
        out = 1.01 * half * (np.abs(one) + np.abs(two)) + (2.0 ** -24 if dtype == "f16" else 0.0)
        terms = 64 + (v if k == 0 else n) / (1 if dtype == "f32" else 16)
        # a root of the sum of squares is what roundings come to; their bound above adds them up
        off = np.abs(one - two)
        assert np.all(off <= err + out + 2 * terms * U32 * size), k
        rms = np.sqrt(np.mean(off ** 2) / np.mean(two ** 2))
        assert rms <= (4 * half if dtype == "f16" else 1e-5), (k, rms)
