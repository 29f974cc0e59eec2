"""The operators at both ends of a tied model together, as its training step uses them: embedding, layer norm, the
head's log-probabilities (or loss) with the embedding as their weight, a 4-bit copy of it as the frozen reference, the
policy loss, and the gradients down to the shared weight.

Each operator has its own numerical tests; here the step's gradients have to be, bit for bit, those of the operators
called one after the other, and each stage's values have to be near the fp64 ones of its own inputs (the bounds of
test_gpu_norm.py and test_gpu_mxfp4.py)."""
import numpy as np
import pytest

from oracle import ends_oracle as eo
from oracle import mx_oracle as mo
from test_gpu_mxfp4 import _check
from test_gpu_norm import U, bounds, compare, np64

pytestmark = pytest.mark.gpu
S, L, H, V = 6, 50, 128, 900


def _model(seed=1, pdtype="float32"):
    import torch
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, H, generator=g) * 0.15).to(torch.bfloat16).cuda()
    gain = (1 + 0.2 * torch.randn(H, generator=g)).to(getattr(torch, pdtype)).cuda()
    shift = (0.1 * torch.randn(H, generator=g)).to(getattr(torch, pdtype)).cuda()
    ids = torch.randint(0, V, (S * L,), generator=g)
    ids[torch.rand(S * L, generator=g) < 0.3] = 7                       # a frequent token
    mask = torch.rand(S, L, generator=g) < 0.8
    targets = torch.randint(0, V, (S * L,), generator=g)
    targets[~mask.reshape(-1)] = -100
    ids[~mask.reshape(-1)] = -100
    adv = torch.randn(S, generator=g)
    return w, gain, shift, ids.cuda(), targets.cuda(), mask.cuda(), adv.cuda()


def _leaves(*tensors):
    return [t.clone().requires_grad_(True) for t in tensors]


def _forward(flce, w, gain, shift, ids, targets):
    x = flce.embedding(ids, w, scale=H ** 0.5)
    y = flce.layer_norm(x, gain, shift)
    return x, y, flce.token_logprobs(y, w, targets, return_entropy=True)


@pytest.mark.parametrize("pdtype", ["float32", "bfloat16"])
def test_policy_step_of_a_tied_model(flce_lib, pdtype):
    import torch
    w, gain, shift, ids, targets, mask, adv = _model(pdtype=pdtype)
    q, s = flce_lib.quantize_mxfp4(w)
    leaves = _leaves(w, gain, shift)
    x, y, (lp, ent) = _forward(flce_lib, *leaves, ids, targets)
    ref = flce_lib.token_logprobs_mxfp4(y.detach(), q, s, targets).view(S, L)
    old = lp.detach().view(S, L) + 0.1 * torch.randn(S, L, generator=torch.Generator().manual_seed(2)).cuda()
    loss = flce_lib.policy_loss(lp.view(S, L), old, adv, ref_logps=ref, entropy=ent.view(S, L), mask=mask, kl_coef=0.05,
                                entropy_coef=0.01)
    got = torch.autograd.grad(loss, leaves)

    # the same, one operator after the other
    lp2, ent2 = (t.detach().view(S, L).requires_grad_(True) for t in (lp, ent))
    again = flce_lib.policy_loss(lp2, old, adv, ref_logps=ref, entropy=ent2, mask=mask, kl_coef=0.05, entropy_coef=0.01)
    g_lp, g_ent = torch.autograd.grad(again, (lp2, ent2))
    hid, head = _leaves(y.detach(), w)
    g_y, g_head = torch.autograd.grad(flce_lib.token_logprobs(hid, head, targets, return_entropy=True), (hid, head),
                                      (g_lp.view(-1), g_ent.view(-1)))
    states, a, b = _leaves(x.detach(), gain, shift)
    g_x, g_gain, g_shift = torch.autograd.grad(flce_lib.layer_norm(states, a, b), (states, a, b), g_y)
    g_embed = flce_lib.embedding_backward(g_x, ids, V, scale=H ** 0.5)
    assert torch.equal(again, loss) and torch.equal(got[1], g_gain) and torch.equal(got[2], g_shift)
    assert torch.equal(got[0], g_head + g_embed)
    assert all(t.isfinite().all() for t in got) and got[0].any()

    # each stage against fp64 on its own inputs
    E = np64(w)
    want = eo.embedding(ids.cpu().numpy(), E, H ** 0.5)
    assert np.all(np.abs(np64(x) - want) <= (2.0 ** -8 + 2 * U) * np.abs(want) + 1e-30)
    (want, tol), *_ = bounds(np64(x), np64(gain), np64(shift), np.zeros((S * L, H)), 1e-5, "bfloat16", pdtype)
    compare(y, want, tol, "hidden")
    _check(np64(ref).reshape(-1), *_entropies(flce_lib, y, q, s, targets), mo.values(*mo.quantize(np64(y))),
           mo.values(*mo.quantize(E)), None, targets.cpu().numpy())


def _entropies(flce, y, q, s, targets):
    return (np64(flce.token_logprobs_mxfp4(y.detach(), q, s, targets, return_entropy=True)[1]),)


@pytest.mark.parametrize("buffer", ["f32", "bf16"])
def test_one_buffer_for_a_tied_weight(flce_lib, buffer):
    """backward's grad_weight buffer takes the embedding's gradient too: in fp32 the sum of both within the last
    additions' rounding, in bf16 one more rounding than autograd's sum of two."""
    import torch
    w, gain, shift, ids, targets, _, _ = _model(3)
    x = flce_lib.embedding(ids, w)
    leaf, a, b = _leaves(x, gain, shift)
    y = flce_lib.layer_norm(leaf, a, b)
    one = torch.ones(1, device="cuda")
    loss, lse, _ = flce_lib.forward(y.detach(), w, targets, reduction="mean")
    gh, gw, _ = flce_lib.backward(y.detach(), w, targets, lse, one, reduction="mean", grad_weight_dtype=buffer)
    g_x, g_gain, g_shift = torch.autograd.grad(y, (leaf, a, b), gh)
    alone = flce_lib.embedding_backward(g_x, ids, V, grad_weight_dtype="f32")
    shared = gw.clone()
    assert flce_lib.embedding_backward(g_x, ids, V, grad_weight=shared) is shared
    sum64 = gw.double() + alone.double()
    half = 2.0 ** -24 if buffer == "f32" else 2.0 ** -8
    assert ((shared.double() - sum64).abs() <= half * sum64.abs() + 3 * U * (gw.double().abs() + alone.double().abs())).all()
    # autograd's own sum of the two for the loss as one op
    tied, a2, b2 = _leaves(w, gain, shift)
    total = flce_lib.linear_cross_entropy(flce_lib.layer_norm(flce_lib.embedding(ids, tied), a2, b2), tied, targets,
                                          reduction="mean")
    got = torch.autograd.grad(total, (tied, a2, b2))
    assert torch.equal(total, loss) and torch.equal(got[1], g_gain) and torch.equal(got[2], g_shift)
    twice = 2.0 ** -8 * (gw.double().abs() + alone.double().abs() + sum64.abs())
    assert ((got[0].double() - sum64).abs() <= twice + half * gw.double().abs() + 3 * U).all()


def test_the_step_as_a_graph(flce_lib):
    """Captured whole and replayed on other tokens, against eager steps in between."""
    import torch
    w, gain, shift, ids, targets, mask, adv = _model(5)
    q, s = flce_lib.quantize_mxfp4(w)
    leaves = _leaves(w, gain, shift)
    old = torch.full((S, L), -5.0, device="cuda")

    def step():
        _, y, (lp, ent) = _forward(flce_lib, *leaves, ids, targets)
        ref = flce_lib.token_logprobs_mxfp4(y.detach(), q, s, targets).view(S, L)
        loss = flce_lib.policy_loss(lp.view(S, L), old, adv, ref_logps=ref, entropy=ent.view(S, L), mask=mask,
                                    kl_coef=0.05, entropy_coef=0.01)
        return (loss.detach(), *torch.autograd.grad(loss, leaves))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        ids.copy_(torch.randint(0, V, (S * L,), generator=torch.Generator().manual_seed(10 + k)))
        graph.replay()
        torch.cuda.synchronize()
        for p, r in zip(out, step()):
            assert torch.equal(p, r)


def test_recomputed_in_the_backward_pass(flce_lib):
    """Under activation checkpointing, and with what the operators save packed to the host: the same gradients."""
    import torch
    from torch.utils.checkpoint import checkpoint
    w, gain, shift, ids, targets, _, _ = _model(7)

    def grads(how):
        leaves = _leaves(w, gain, shift)
        loss = how(lambda a, b, c: _forward(flce_lib, a, b, c, ids, targets)[2][0].sum(), leaves)
        return (loss.detach(), *torch.autograd.grad(loss, leaves))

    def packed(f, leaves):
        with torch.autograd.graph.save_on_cpu():
            return f(*leaves)

    want = grads(lambda f, leaves: f(*leaves))
    for how in (lambda f, leaves: checkpoint(lambda *a: f(*a), *leaves, use_reentrant=False), packed):
        for p, r in zip(grads(how), want):
            assert torch.equal(p, r)


def test_steps_on_two_threads(flce_lib):
    """Two threads, each with its own stream, model and library calls, at the same time: neither's results change."""
    import threading

    import torch
    problems = [_model(seed) for seed in (11, 12)]
    problems = [(*p, *flce_lib.quantize_mxfp4(p[0])) for p in problems]

    def step(p):
        w, gain, shift, ids, targets, _, _, q, s = p
        leaves = _leaves(w, gain, shift)
        _, y, (lp, _) = _forward(flce_lib, *leaves, ids, targets)
        return (flce_lib.token_logprobs_mxfp4(y.detach(), q, s, targets), lp.detach(),
                *torch.autograd.grad(lp.sum(), leaves))

    want = [step(p) for p in problems]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[k] += [step(problems[k]) for _ in range(20)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for k in (0, 1):
        assert len(got[k]) == 20
        for out in got[k]:
            for p, r in zip(out, want[k]):
                assert torch.equal(p, r)
