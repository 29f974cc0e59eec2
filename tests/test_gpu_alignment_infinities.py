"""Losses over infinite log-probabilities, which token_logprobs gives for a target that its bias masks."""
import math

import pytest

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
INF = math.inf


def _pair_loss(h, eps):
    """-(1 - eps) log sigmoid(h) - eps log sigmoid(-h); a term of weight 0 is none."""
    def minus_log_sigmoid(x):
        return max(-x, 0.0) + math.log1p(math.exp(-abs(x)))
    return ((1 - eps) * minus_log_sigmoid(h) if eps < 1 else 0.0) + (eps * minus_log_sigmoid(-h) if eps else 0.0)


def _pair_slope(h, eps):
    def sigmoid(x):
        return 1 / (1 + math.exp(-x)) if x > -700 else 0.0
    return -(1 - eps) * sigmoid(-h) + eps * sigmoid(h)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("eps", [0.0, 0.1, 0.5, 1.0])
def test_smoothed_sigmoid_at_infinite_margins(packed, eps):
    """The chosen answer of pair 0 has probability 0, the rejected one of pair 1; pairs 2 to 4 are finite."""
    import torch
    import linear_cross_entropy_tiled_amd as flce
    length, pairs, beta = 6, 5, 0.25
    x = -torch.arange(1, 2 * pairs * length + 1, dtype=torch.float32).reshape(2 * pairs, length) / 16
    x[0, 2] = -INF
    x[pairs + 1, 5] = -INF
    x[2] -= 40.0
    sums = x.double().sum(1)
    h = [beta * float(sums[p] - sums[pairs + p]) for p in range(pairs)]
    assert h[0] == -INF and h[1] == INF and all(map(math.isfinite, h[2:]))
    want = [_pair_loss(v, eps) for v in h]
    assert not any(map(math.isnan, want))

    offsets = torch.arange(0, 2 * pairs * length + 1, length, device="cuda") if packed else None
    lp = (x.reshape(-1) if packed else x).cuda().requires_grad_(True)

    def call(reduction):
        return flce.preference_loss(lp, offsets=offsets, beta=beta, label_smoothing=eps, reduction=reduction)

    # sums of dyadic numbers are exact, the rest is fp64 and one rounding to fp32
    got = call("none")
    for v, w in zip(got.tolist(), want):
        assert v == w if math.isinf(w) else abs(v - w) <= 2 * U32 * abs(w) + 2.0 ** -126, (v, w)
    for reduction, share in (("sum", 1.0), ("mean", 1 / pairs)):
        v, w = float(call(reduction)), sum(want) * share
        assert v == w if math.isinf(w) else abs(v - w) <= 2 * U32 * abs(w), (reduction, v, w)
        grad, = torch.autograd.grad(call(reduction), (lp,))
        grad = grad.reshape(2 * pairs, length).double().cpu()
        for p in range(pairs):
            d = _pair_slope(h[p], eps) * beta * share
            # fp64 (whose 1 - eps has an absolute error), rounded to fp32, times an upstream 1
            assert (grad[p] - d).abs().max() <= 2 * U32 * abs(d) + 2.0 ** -50
            assert (grad[pairs + p] + d).abs().max() <= 2 * U32 * abs(d) + 2.0 ** -50
