"""What token_logprobs_int8 takes: scales and biases that begin anywhere, the whole range of hidden sizes that
int32 sums allow, whatever params->dtype says."""
import numpy as np
import pytest

import linear_cross_entropy_tiled_amd as flce


@pytest.mark.parametrize("h", [16, 4096, 16384, 32768, 65536, 1 << 17])
@pytest.mark.parametrize("v", [1000, 33000, 128256])
def test_sizes_do_not_depend_on_the_gradients_fields(h, v):
    sizes = {flce.flce_logprobs_int8_workspace_size(flce.make_params(n, h, v, reduction="none", **opts))
             for n in (100,) for opts in (dict(dtype="bf16"), dict(dtype="f16"), dict(dtype="f32"),
                                          dict(vocab_chunk=256), dict(dtype="f32", vocab_chunk=65536))}
    assert len(sizes) == 1


def test_most_tokens():
    """N H < 2^30 and N <= 2^22 - 256, for every dtype."""
    assert flce.flce_logprobs_int8_workspace_size(flce.make_params((1 << 22) - 256, 16, 1000, reduction="none", dtype="f32"))
    for dtype in ("bf16", "f32"):
        flce.flce_logprobs_int8_workspace_size(flce.make_params((1 << 18) - 1, 4096, 1000, reduction="none", dtype=dtype))
        with pytest.raises(flce.FlceError) as e:
            flce.flce_logprobs_int8_workspace_size(flce.make_params(1 << 18, 4096, 1000, reduction="none", dtype=dtype))
        assert e.value.code == flce.FLCE_ERR_UNSUPPORTED


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


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 100, 1000])
def test_long_hidden_states_and_a_long_vocabulary(flce_lib, n):
    """A weight of 4.3 GB: its rows' offsets pass 32 bits, in narrow, small and large tiles.  The error is that of
    test_gpu_logprobs_int8.py."""
    import torch
    h, v, u32 = 1 << 17, 33000, 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(n)
    wq = torch.randint(-127, 128, (v, h), generator=g, device="cuda", dtype=torch.int8)
    q = torch.randint(-127, 128, (n, h), generator=g, device="cuda", dtype=torch.int8)
    s = (0.5 + torch.rand(n, generator=g, device="cuda")) * 2.0 ** -10
    ws = (0.5 + torch.rand(v, generator=g, device="cuda")) * 2.0 ** -10
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[0], t[-1] = v - 1, 16384       # the last row, and the first beyond 2^31 bytes
    lp, ent = flce_lib.token_logprobs_int8(q, wq, ws, t, hidden_scale=s, return_entropy=True)
    qd = q.double()
    product = torch.cat([qd @ wq[i:i + 1000].double().t().contiguous() for i in range(0, v, 1000)], 1)
    z = product * s.double()[:, None] * ws.double()
    l = z - torch.logsumexp(z, 1, keepdim=True)
    ez = 5 * u32 * z.abs().amax(1)
    own = 24 * u32 * (z.abs().amax(1) + np.log(v) + 1)
    spread = 1 + 2 * (z.amax(1) - z.amin(1) + np.log(v))
    want = l.gather(1, t[:, None])[:, 0]
    assert ((lp.double() - want).abs() <= 2 * ez + own).all()
    assert ((ent.double() + (l.exp() * l).sum(1)).abs() <= spread * ez + 2 * own).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [(1 << 22) + 1, (1 << 24) + 3])
def test_quantize_many_rows(flce_lib, rows):
    """More rows than one launch has workgroups for."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, 16, generator=g, device="cuda", dtype=torch.bfloat16)
    x[-1, 3], x[5] = float("nan"), 0.0
    q, scale = flce_lib.quantize_int8(x)
    for at in range(0, rows, 1 << 21):       # the definition, in fp32
        v = x[at:at + (1 << 21)].float()
        top = v.abs().amax(1)
        s = top * torch.tensor(1.0 / 127.0, device="cuda")
        live = top >= 1e-30                  # NaN is not
        r = torch.where(live, 1.0 / s, 0.0)
        want = torch.where(live[:, None], torch.round(v * r[:, None]), 0.0).to(torch.int8)
        assert torch.equal(q[at:at + (1 << 21)], want)
        got = scale[at:at + (1 << 21)]
        assert torch.equal(torch.isnan(got), torch.isnan(top))
        assert torch.equal(torch.nan_to_num(got), torch.where(live, s, 0.0))
