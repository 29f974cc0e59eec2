"""token_logprobs and its C entry points refuse what the kernels cannot take (CPU only)."""
import pytest
import torch

import linear_cross_entropy_tiled_amd as flce

N, H, V = 16, 64, 100


@pytest.mark.parametrize("change,exc", [
    ({}, ValueError),                                                        # consistent, but on the CPU
    (dict(weight=torch.zeros(V, H)), TypeError),
    (dict(weight=torch.zeros(V, H + 8, dtype=torch.bfloat16)), ValueError),
    (dict(targets=torch.zeros(N)), TypeError),
    (dict(targets=torch.zeros(N + 1, dtype=torch.int64)), ValueError),
    (dict(bias=torch.zeros(V - 1, dtype=torch.bfloat16)), ValueError),
    (dict(hidden=torch.zeros(2, 8, H, dtype=torch.bfloat16)), ValueError),
    (dict(hidden=torch.zeros(H, N, dtype=torch.bfloat16).t()), ValueError),
])
def test_token_logprobs_rejects(change, exc):
    a = dict(hidden=torch.zeros(N, H, dtype=torch.bfloat16), weight=torch.zeros(V, H, dtype=torch.bfloat16),
             targets=torch.zeros(N, dtype=torch.int64), bias=None)
    a.update(change)
    with pytest.raises(exc):
        flce.token_logprobs(a["hidden"], a["weight"], a["targets"], a["bias"])


def test_abi_codes():
    bad, odd = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED
    for opts, code in ((dict(reduction="sum"), bad), (dict(z_loss=0.1), bad), (dict(hidden=12), odd)):
        h = opts.pop("hidden", H)
        p = flce.make_params(N, h, V, **{"reduction": "none", **opts})
        with pytest.raises(flce.FlceError) as e:
            flce.flce_logprobs_workspace_size(p, 0)
        assert e.value.code == code
        assert flce.flce_logprobs_forward(p, 16, 16, None, 16, 16, None, 16, 16, 1 << 30, None) == code
    p = flce.make_params(N, H, V, reduction="none")
    with pytest.raises(flce.FlceError):
        flce.flce_logprobs_workspace_size(p, 2)
    need = [flce.flce_logprobs_workspace_size(p, k) for k in (0, 1)]
    assert need[1] > flce.flce_workspace_size(p, 1)

    def fwd(x=16, w=16, b=None, t=16, lp=16, ent=None, lse=16, ws=16, n=need[0]):
        return flce.flce_logprobs_forward(p, x, w, b, t, lp, ent, lse, ws, n, None)

    def bwd(x=16, w=16, b=None, t=16, lse=16, ent=16, g=16, e=16, gx=16, gw=16, gb=None, ws=16, n=need[1]):
        return flce.flce_logprobs_backward(p, x, w, b, t, lse, ent, g, e, gx, gw, gb, ws, n, None)

    for name in ("x", "w", "t", "lp", "lse", "ws"):
        assert fwd(**{name: None}) == bad, name
    for name in ("x", "w", "t", "lse", "ent", "ws"):
        assert bwd(**{name: None}) == bad, name
    assert bwd(gb=16) == bad                     # a bias gradient without a bias
    for name in ("x", "w", "b", "ws"):
        assert fwd(**{name: 24}) == odd and bwd(**{name: 24}) == odd, name
    assert fwd(t=20) == odd and bwd(t=20) == odd         # int64 values
    assert fwd(lp=18) == odd and fwd(lse=18) == odd and bwd(g=18) == odd and bwd(e=18) == odd
    assert fwd(n=need[0] - 1) == flce.FLCE_ERR_WORKSPACE_TOO_SMALL
    assert bwd(n=need[1] - 1) == flce.FLCE_ERR_WORKSPACE_TOO_SMALL
