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
