"""torch.jit.trace of the ends of a model: a recorded graph gives the eager call's results, also when nothing of the
call that it was recorded from is there any more."""
import gc

import pytest

pytestmark = pytest.mark.gpu


def _trace(fn, args):
    import torch
    return torch.jit.trace(fn, args, check_trace=False)


@pytest.mark.parametrize("opts", [{}, dict(logit_scale=0.5, softcap=3.0, ignore_index=7)])
def test_scores(flce_lib, opts):
    import torch
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(40, 96, device="cuda", generator=g).bfloat16()
    q, s = flce_lib.quantize_mxfp4(torch.randn(300, 96, device="cuda", generator=g))
    bias = torch.randn(300, device="cuda", generator=g)
    t = torch.randint(0, 300, (40,), device="cuda", generator=g)
    traced = _trace(lambda x, t: flce_lib.token_logprobs_mxfp4(x, q, s, t, bias, **opts), (x, t))
    from linear_cross_entropy_tiled_amd import logprobs
    for f in vars(logprobs).values():                 # nothing is left of the recorded call
        if hasattr(f, "cache_clear"):
            f.cache_clear()
    gc.collect()
    for seed in range(3):
        g.manual_seed(seed)
        x = torch.randn(40, 96, device="cuda", generator=g).bfloat16()
        t = torch.randint(0, 300, (40,), device="cuda", generator=g)
        assert torch.equal(traced(x, t), flce_lib.token_logprobs_mxfp4(x, q, s, t, bias, **opts))


def test_embedding_and_layer_norm(flce_lib):
    import torch
    g = torch.Generator("cuda").manual_seed(2)
    w = torch.randn(50, 72, device="cuda", generator=g)
    gain = torch.randn(72, device="cuda", generator=g)

    def fn(ids):
        return flce_lib.layer_norm(flce_lib.embedding(ids, w, scale=2.0), gain, eps=1e-3)

    ids = torch.randint(0, 50, (20,), device="cuda", generator=g)
    traced = _trace(fn, (ids,))
    assert torch.equal(traced(ids.flip(0)), fn(ids.flip(0)))
    assert torch.equal(traced(ids[:7]), fn(ids[:7]))               # fewer rows of the recorded types are no other call


def test_other_sizes_than_the_recorded_ones(flce_lib):
    """Where the recorded graph's constants do not fit, the call is refused, not made."""
    import torch
    gain, ids = torch.ones(64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    norm = _trace(lambda x: flce_lib.layer_norm(x, gain), (torch.randn(4, 64, device="cuda"),))
    for x in (torch.randn(4, 128, device="cuda"), torch.randn(4, 32, device="cuda"), torch.randn(4, 64, device="cuda").double()):
        with pytest.raises(RuntimeError, match="type, size, layout or device"):
            norm(x)
    q, s = flce_lib.quantize_mxfp4(torch.randn(30, 64, device="cuda"))
    scores = _trace(lambda x: flce_lib.token_logprobs_mxfp4(x, q, s, ids), (torch.randn(4, 64, device="cuda"),))
    for shape in ((4, 128), (5, 64), (3, 64)):
        with pytest.raises(RuntimeError, match="type, size, layout or device"):
            scores(torch.randn(*shape, device="cuda"))
    lookup = _trace(lambda w: flce_lib.embedding(ids, w), (torch.randn(10, 64, device="cuda"),))
    w = torch.randn(7, 40, device="cuda")
    assert torch.equal(lookup(w), w[ids])                          # a table of any size fits


def _by_pointer(flce_lib):
    """name -> (function, its argument): calls that are no recorded operator."""
    import torch
    g = torch.Generator("cuda").manual_seed(4)
    n, h, v = 64, 96, 300
    x = torch.randn(n, h, device="cuda", generator=g).bfloat16()
    w = torch.randn(v, h, device="cuda", generator=g).bfloat16()
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    one, adv = torch.ones(1, device="cuda"), torch.ones(4, device="cuda")
    lp = -torch.rand(4, 16, device="cuda", generator=g)
    lse = flce_lib.forward(x, w, t, reduction="mean")[1]
    q, s = flce_lib.quantize_int8(w)
    target, rows, columns = torch.zeros(n, v, device="cuda"), torch.ones(n, device="cuda"), torch.ones(v, device="cuda")
    return {
        "forward": (lambda x: flce_lib.forward(x, w, t, reduction="mean")[0], x),
        "backward": (lambda x: flce_lib.backward(x, w, t, lse, one, reduction="mean")[0], x),
        "forward_backward": (lambda x: flce_lib.forward_backward(x, w, t, one, reduction="mean")[0], x),
        "weighted_mse": (lambda x: flce_lib.weighted_mse(x, w, target, rows, columns)[0], x),
        "token_logprobs": (lambda x: flce_lib.token_logprobs(x, w, t), x),
        "quantize_int8": (lambda x: flce_lib.quantize_int8(x)[0], x),
        "token_logprobs_int8": (lambda x: flce_lib.token_logprobs_int8(x, q, s, t), x),
        "policy_loss": (lambda lp: flce_lib.policy_loss(lp, lp - 0.1, adv), lp),
        "preference_loss": (lambda lp: flce_lib.preference_loss(lp, lp - 0.1), lp),
        "embedding_backward": (lambda x: flce_lib.embedding_backward(x, t, v), x),
    }


@pytest.mark.parametrize("name", ["forward", "backward", "forward_backward", "weighted_mse", "token_logprobs",
                                  "quantize_int8", "token_logprobs_int8", "policy_loss", "preference_loss",
                                  "embedding_backward"])
def test_a_call_by_pointers_is_not_recorded(flce_lib, name):
    """It would be replayed as the allocation of its outputs, without the call that fills them."""
    fn, a = _by_pointer(flce_lib)[name]
    fn(a)
    with pytest.raises(RuntimeError, match="cannot be recorded"):
        _trace(fn, (a,))
    with pytest.raises(RuntimeError, match="cannot be recorded"):
        _trace(fn, (a.clone().requires_grad_(True),))


@pytest.mark.parametrize("one_pass", [False, True])
def test_the_loss_as_a_recorded_function(flce_lib, one_pass):
    """Autograd's functions are recorded as themselves; this one looks at its tensors' sizes in each call."""
    import torch
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(64, 96, device="cuda", generator=g).bfloat16()
    w = torch.randn(300, 96, device="cuda", generator=g).bfloat16()
    t = torch.randint(0, 300, (64,), device="cuda", generator=g)

    def loss(x, w):
        return flce_lib.linear_cross_entropy(x, w, t, reduction="mean", one_pass=one_pass)

    traced = _trace(loss, (x, w))
    for other in (x * 0.5, -x):
        assert torch.equal(traced(other, w), loss(other, w))
    with pytest.raises((RuntimeError, ValueError)):
        traced(x[:10], w)                                          # 64 targets, 10 rows
    leaf = x.clone().requires_grad_(True)
    got, = torch.autograd.grad(_trace(loss, (leaf, w))(leaf, w), leaf)
    assert torch.equal(got, torch.autograd.grad(loss(leaf, w), leaf)[0])
