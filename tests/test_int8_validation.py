"""quantize_int8, token_logprobs_int8 and their C entry points refuse what the kernels cannot
take (CPU only)."""
import pytest
import torch

import linear_cross_entropy_tiled_amd as flce

N, H, V = 16, 64, 100


@pytest.mark.parametrize("change,exc", [
    ({}, ValueError),                                                        # consistent, but on the CPU
    (dict(weight=torch.zeros(V, H)), TypeError),
    (dict(weight=torch.zeros(V, H + 16, dtype=torch.int8)), ValueError),
    (dict(hidden=torch.zeros(N, H, dtype=torch.int8)), TypeError),           # without its scale
    (dict(hidden_scale=torch.zeros(N)), TypeError),                          # a scale for unquantized states
    (dict(hidden=torch.zeros(N, H, dtype=torch.int8), hidden_scale=torch.zeros(N + 1)), ValueError),
    (dict(hidden=torch.zeros(N, 56), weight=torch.zeros(V, 56, dtype=torch.int8)), ValueError),
    (dict(weight_scale=torch.zeros(V, dtype=torch.bfloat16)), TypeError),
    (dict(weight_scale=torch.zeros(V, 1)), ValueError),
    (dict(bias=torch.zeros(V, dtype=torch.bfloat16)), TypeError),
    (dict(targets=torch.zeros(N)), TypeError),
    (dict(targets=torch.zeros(N - 1, dtype=torch.int64)), ValueError),
    (dict(hidden=torch.zeros(H, N).t()), ValueError),
    (dict(hidden=torch.zeros(N, H, dtype=torch.float64)), TypeError),
])
def test_token_logprobs_int8_rejects(change, exc):
    a = dict(hidden=torch.zeros(N, H), weight=torch.zeros(V, H, dtype=torch.int8), weight_scale=torch.ones(V),
             targets=torch.zeros(N, dtype=torch.int64), bias=None, hidden_scale=None)
    a.update(change)
    with pytest.raises(exc):
        flce.token_logprobs_int8(a["hidden"], a["weight"], a["weight_scale"], a["targets"], a["bias"],
                                 hidden_scale=a["hidden_scale"])


@pytest.mark.parametrize("x,exc", [
    (torch.zeros(4, 16), ValueError), (torch.zeros(4, 24), ValueError), (torch.zeros(4, 0), ValueError),
    (torch.zeros(64), ValueError), (torch.zeros(16, 32).t(), ValueError), (torch.zeros(4, 16, dtype=torch.int8), TypeError),
])
def test_quantize_int8_rejects(x, exc):
    with pytest.raises(exc):
        flce.quantize_int8(x)


def test_abi_codes():
    bad, odd = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED
    for a, code in (((3, 16, 4, 16, 16, 16), bad), ((1, 16, -1, 16, 16, 16), bad), ((1, 16, 4, 0, 16, 16), bad),
                    ((1, None, 4, 16, 16, 16), bad), ((1, 16, 4, 16, None, 16), bad), ((1, 16, 4, 16, 16, None), bad),
                    ((1, 16, 4, 24, 16, 16), odd), ((1, 24, 4, 16, 16, 16), odd), ((1, 16, 4, 16, 24, 16), odd),
                    ((1, 16, 4, 16, 16, 18), odd), ((1, 16, 1 << 31, 16, 16, 16), odd)):
        assert flce.flce_quantize_int8(*a, None) == code, a
    for opts, code in ((dict(reduction="sum"), bad), (dict(z_loss=0.1), bad), (dict(h=72), odd), (dict(h=(1 << 17) + 16), odd)):
        h = opts.pop("h", H)
        p = flce.make_params(N, h, V, **{"reduction": "none", **opts})
        with pytest.raises(flce.FlceError) as e:
            flce.flce_logprobs_int8_workspace_size(p)
        assert e.value.code == code
        assert flce.flce_logprobs_int8(p, 16, 16, 16, 16, None, 16, 16, None, 16, 16, 1 << 30, None) == code
    p = flce.make_params(N, H, V, reduction="none")
    need = flce.flce_logprobs_int8_workspace_size(p)

    def call(x=16, s=16, w=16, ws=16, b=None, t=16, lp=16, lse=16, work=16, n=need):
        return flce.flce_logprobs_int8(p, x, s, w, ws, b, t, lp, None, lse, work, n, None)

    for name in ("x", "s", "w", "ws", "t", "lp", "lse", "work"):
        assert call(**{name: None}) == bad, name
    for name in ("x", "w", "ws", "b", "work"):
        assert call(**{name: 24}) == odd, name
    assert call(s=18) == odd and call(t=20) == odd and call(lp=18) == odd and call(n=need - 1) == flce.FLCE_ERR_WORKSPACE_TOO_SMALL
