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


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("reduction", ["mean", "sequence_mean", "sum", "none"])
def test_terms_with_coefficient_zero_add_nothing(dtype, reduction):
    """A reference given for its metric alone, and entropies without a coefficient, leave loss and gradient as
    they are without them, whatever they hold."""
    import torch
    import linear_cross_entropy_tiled_amd as flce
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(5)
    s, length = 3, 301
    lp = torch.log(torch.rand(s, length, generator=g).clamp_min(1e-3))
    old = (lp + 0.3 * torch.randn(s, length, generator=g)).to(dt).cuda()
    ref = lp + 0.3 * torch.randn(s, length, generator=g)
    ent = torch.rand(s, length, generator=g)
    lp[0, 7] = -INF                              # ratio 0, ref - logp infinite
    lp[2, 300] = -120.0                          # e^(ref - logp) overflows fp32
    ref[1, 4], ref[1, 290], ref[2, 12] = -INF, INF, math.nan
    ref[2, 300] = -1.0
    ent[0, 0], ent[1, 77], ent[2, 256] = INF, -INF, math.nan
    adv = torch.randn(s, length, generator=g).cuda()
    mask = (torch.rand(s, length, generator=g) < 0.9).cuda()
    mask[0, 7] = mask[1, 4] = mask[1, 290] = mask[2, 300] = mask[2, 12] = True
    mask[0, 0] = mask[1, 77] = mask[2, 256] = True
    lp = lp.to(dt).cuda().requires_grad_(True)
    ent = ent.to(dt).cuda().requires_grad_(True)

    def call(**more):
        out = flce.policy_loss(lp, old, adv, mask=mask, reduction=reduction, return_metrics=True, **more)
        up = torch.ones_like(out[0])
        leaves = (lp, ent) if "entropy" in more else (lp,)
        return (*out, torch.autograd.grad(out[0], leaves, up))

    loss, metrics, (grad,) = call()
    assert torch.isfinite(loss).all() and torch.isfinite(grad).all()
    for more in (dict(ref_logps=ref.to(dt).cuda()), dict(entropy=ent), dict(ref_logps=ref.to(dt).cuda(), entropy=ent)):
        loss2, metrics2, grads = call(**more)
        assert torch.equal(loss2, loss) and torch.equal(grads[0], grad), list(more)
        if "entropy" in more:
            assert not grads[1].any()
        assert metrics2["num_tokens"] == metrics["num_tokens"] and metrics2["clip_fraction"] == metrics["clip_fraction"]
        if "ref_logps" in more:
            assert torch.isnan(metrics2["kl"])          # the metric says what the reference holds


@pytest.mark.parametrize("ref0,want", [(-INF, INF), (-3.0, None)])
def test_kl_of_a_reference_without_coefficient(ref0, want):
    import torch
    import linear_cross_entropy_tiled_amd as flce
    lp = torch.tensor([[-1.0, -2.0, -3.0]], device="cuda")
    ref = torch.tensor([[-1.5, ref0, -2.0]], device="cuda")
    loss, metrics = flce.policy_loss(lp, lp, torch.ones_like(lp), ref_logps=ref, return_metrics=True)
    assert loss == -1.0
    d = (ref - lp).double()
    want = float((torch.expm1(d) - d).mean()) if want is None else want
    assert float(metrics["kl"]) == want or abs(float(metrics["kl"]) - want) <= 16 * U32 * want
