"""Forward-mode derivatives are refused, not dropped: which calls go through autograd (CPU)."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from linear_cross_entropy_tiled_amd.logprobs import differentiable


def test_tangents_go_through_autograd():
    x, y = torch.zeros(3), torch.zeros(3)
    assert not differentiable(x, y, None)
    with fwAD.dual_level():
        d = fwAD.make_dual(x, torch.ones(3))
        assert not d.requires_grad
        assert differentiable(d) and differentiable(y, None, d) and differentiable(d.view(3, 1))
        assert not differentiable(y, d.detach())
        with torch.no_grad():                  # stops the recording, not the tangents
            assert differentiable(d)
    assert not differentiable(d)               # the level is gone, and its tangents


def test_recorded_calls_go_through_autograd():
    x = torch.zeros(3, requires_grad=True)
    assert differentiable(x) and differentiable(None, x)
    with torch.no_grad():
        assert not differentiable(x)
    assert not differentiable(x.detach())
    with torch.inference_mode():
        assert not differentiable(torch.zeros(3))


@pytest.mark.gpu
@pytest.mark.parametrize("grad_mode", [True, False])
def test_dual_inputs_are_refused(grad_mode):
    import linear_cross_entropy_tiled_amd as flce
    dev, n, h, v, s = "cuda", 8, 16, 40, 2
    hidden, weight, bias = (torch.ones(*k, device=dev) for k in ((n, h), (v, h), (v,)))
    targets = torch.zeros(n, dtype=torch.int64, device=dev)
    q, scale = flce.quantize_int8(weight)
    tok = torch.full((s, n // s), -1.0, device=dev)
    adv = torch.ones(s, n // s, device=dev)

    def dual(x):
        return fwAD.make_dual(x, torch.ones_like(x))

    with torch.set_grad_enabled(grad_mode), fwAD.dual_level():
        for args in ((dual(hidden), weight, targets), (hidden, dual(weight), targets),
                     (hidden, weight, targets, dual(bias))):
            with pytest.raises(NotImplementedError):
                flce.token_logprobs(*args)
        for kw in (dict(hidden=dual(hidden)), dict(weight_scale=dual(scale)), dict(bias=dual(bias))):
            a = dict(hidden=hidden, weight=q, weight_scale=scale, targets=targets, bias=bias)
            with pytest.raises(ValueError, match="no gradient"):
                flce.token_logprobs_int8(**{**a, **kw})
        with pytest.raises(NotImplementedError):
            flce.preference_loss(dual(tok), tok)
        with pytest.raises(NotImplementedError):
            flce.preference_loss(tok, dual(tok))
        for kw in (dict(logps=dual(tok)), dict(entropy=dual(tok)), dict(old_logps=dual(tok)),
                   dict(ref_logps=dual(tok)), dict(advantages=dual(adv))):
            a = dict(logps=tok, old_logps=tok, advantages=adv, ref_logps=tok, entropy=tok)
            with pytest.raises(NotImplementedError):
                flce.policy_loss(**{**a, **kw}, kl_coef=0.1, entropy_coef=0.1)
        # without a tangent the same calls run
        flce.token_logprobs(hidden, weight, targets, bias)
        flce.token_logprobs_int8(hidden, q, scale, targets, bias)
        flce.preference_loss(tok, tok)
        flce.policy_loss(tok, tok, adv, ref_logps=tok, entropy=tok, kl_coef=0.1, entropy_coef=0.1)
