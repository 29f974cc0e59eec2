"""The alignment operators together, as a training step uses them: 8-bit reference scores,
log-probabilities of the policy, the loss, its gradients down to the head; against the
oracle's chain in fp64.

Tolerance: the chain's gradient of a log-probability is within a few 2^-24 of the oracle's
on the same log-probabilities; those move by at most ~1e-5 (test_gpu_token_logprobs.py), and
the loss's second derivative is at most ~2 here, so the logit gradient is off by its own
rounding in bf16 (2^-8 of each entry) and 1e-4 of the row's; the outputs are rounded once
more (2^-8)."""
import numpy as np
import pytest

from oracle import alignment_oracle as ao

pytestmark = pytest.mark.gpu


def _np(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def _batch(seed, s=6, length=50, h=64, v=900):
    import torch
    rng = np.random.default_rng(seed)
    n = s * length
    x = torch.from_numpy(rng.normal(size=(n, h))).to(torch.bfloat16)
    w = torch.from_numpy(rng.normal(size=(v, h)) * 0.15).to(torch.bfloat16)
    t = torch.from_numpy(rng.integers(0, v, size=n))
    mask = torch.from_numpy(rng.random((s, length)) < 0.8)
    t[~mask.reshape(-1)] = -100
    return x, w, t, mask, torch.from_numpy(rng.normal(size=s)).float()


def _close(got, want, a, what):
    """a: sums of the absolute terms of each output."""
    assert np.all(np.abs(_np(got) - want) <= 1.02 * 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2e-4) * a + 1e-7), what


def _abs_terms(X, W, T, g, e):
    logp, ent, z, _ = ao.token_logprobs(X, W, None, T)
    lse = z.max(1) + np.log(np.exp(z - z.max(1, keepdims=True)).sum(1))
    l = z - lse[:, None]
    p = np.exp(l) * (T >= 0)[:, None]
    d = np.abs(g)[:, None] * p + np.abs(e)[:, None] * p * (np.abs(l) + ent[:, None])
    rows = np.flatnonzero(T >= 0)
    d[rows, T[rows]] += np.abs(g)[rows]
    return d @ np.abs(W), d.T @ np.abs(X)


@pytest.mark.parametrize("reduction", ["mean", "sequence_mean"])
def test_policy_step(flce_lib, reduction):
    import torch
    x, w, t, mask, adv = _batch(1)
    wq, ws = flce_lib.quantize_int8(w.cuda())
    tt = t.cuda()
    ref = flce_lib.token_logprobs_int8(x.cuda(), wq, ws, tt).view(mask.shape)
    old = (ref + 0.1 * torch.randn(mask.shape, generator=torch.Generator().manual_seed(1)).cuda())
    hx, hw = x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    lp, ent = flce_lib.token_logprobs(hx, hw, tt, return_entropy=True)
    loss = flce_lib.policy_loss(lp.view(mask.shape), old, adv.cuda(), ref_logps=ref, entropy=ent.view(mask.shape),
                                mask=mask.cuda(), kl_coef=0.1, entropy_coef=0.02, reduction=reduction)
    loss.backward()
    X, W, T = _np(x), _np(w), t.numpy()
    want = ao.policy(_np(lp).reshape(mask.shape), _np(old), adv.numpy(), _np(ref), _np(ent).reshape(mask.shape), None,
                     mask.numpy(), kl_coef=0.1, entropy_coef=0.02, reduction=reduction)
    assert abs(loss.item() - want["loss"]) <= 1e-5
    g, e = want["grad"](1.0).reshape(-1), want["grad_entropy"](1.0).reshape(-1)
    gx, gw, _ = ao.token_logprobs_grads(X, W, None, T, g, e)
    ax, aw = _abs_terms(X, W, T, g, e)
    _close(hx.grad, gx, ax, "hidden")
    _close(hw.grad, gw, aw, "weight")


def test_preference_step_and_accumulated_backward(flce_lib):
    import torch
    x, w, t, mask, _ = _batch(2)
    hx, hw = x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    lens = mask.sum(1)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    flat = torch.nonzero(mask.reshape(-1))[:, 0]
    T = t[flat]
    with torch.no_grad():
        ref = flce_lib.token_logprobs(hx[flat.cuda()], hw * 0.9, T.cuda())

    def step():
        lp = flce_lib.token_logprobs(hx[flat.cuda()], hw, T.cuda())
        return lp, flce_lib.preference_loss(lp, ref, offsets=off.cuda(), beta=0.05)

    lp, loss = step()
    loss.backward()
    first = [hx.grad.clone(), hw.grad.clone()]
    step()[1].backward()          # a second step adds to the leaves' gradients
    assert torch.equal(hw.grad, (first[1].float() * 2).bfloat16())
    _, _, grad = ao.preference(_np(lp), _np(ref), off.numpy(), None, beta=0.05)
    g = grad(1.0)
    X, W = _np(x)[flat], _np(w)
    gx, gw, _ = ao.token_logprobs_grads(X, W, None, T.numpy(), g, 0 * g)
    ax, aw = _abs_terms(X, W, T.numpy(), g, 0 * g)
    _close(first[0][flat.cuda()], gx, ax, "hidden")
    _close(first[1], gw, aw, "weight")


def test_a_training_step_in_a_graph(flce_lib):
    """Forward and backward of the whole chain captured and replayed, with new contents in between."""
    import torch
    x, w, t, mask, adv = _batch(3)
    wq, ws = flce_lib.quantize_int8(w.cuda())
    hx, hw = x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    tt, m, a = t.cuda(), mask.cuda(), adv.cuda()
    old = flce_lib.token_logprobs_int8(x.cuda() * 1.05, wq, ws, tt).view(mask.shape)

    def step():
        ref = flce_lib.token_logprobs_int8(hx.detach(), wq, ws, tt).view(mask.shape)
        lp, ent = flce_lib.token_logprobs(hx, hw, tt, return_entropy=True)
        loss = flce_lib.policy_loss(lp.view(mask.shape), old, a, ref_logps=ref, entropy=ent.view(mask.shape), mask=m,
                                    kl_coef=0.1, entropy_coef=0.02)
        return [loss.detach(), *torch.autograd.grad(loss, (hx, hw))]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(6):
        with torch.no_grad():
            hx.mul_(0.97)
        want = step()
        for o in outs:
            o.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want)), rep
