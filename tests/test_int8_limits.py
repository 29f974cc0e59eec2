"""What token_logprobs_int8 takes: scales and biases that begin anywhere."""
import pytest


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 16, 70, 300])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_a_vocabulary_slice(flce_lib, n, first):
    """Scales and biases from an odd row on give the bits of aligned copies."""
    import torch
    g = torch.Generator().manual_seed(n + first)
    h, v = 64, 1203
    x = torch.randn(n, h, generator=g).to(torch.bfloat16).cuda()
    q, scale = flce_lib.quantize_int8(torch.randn(v, h, generator=g).cuda())
    b = torch.randn(v, generator=g).cuda()
    t = torch.randint(0, v - first, (n,), generator=g).cuda()
    for bias in (None, b[first:]):
        got = flce_lib.token_logprobs_int8(x, q[first:], scale[first:], t, bias, return_entropy=True)
        want = flce_lib.token_logprobs_int8(x, q[first:], scale[first:].clone(), t,
                                            None if bias is None else bias.clone(), return_entropy=True)
        assert scale[first:].data_ptr() % 16 and all(torch.equal(a, c) for a, c in zip(got, want))
