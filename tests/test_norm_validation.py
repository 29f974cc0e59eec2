"""layer_norm and its C entry points refuse what the kernels cannot take; its fp64 definition against
differences (CPU only)."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_tiled_amd as flce
from oracle import ends_oracle as eo

N, H = 4, 24


@pytest.mark.parametrize("change,exc", [
    ({}, ValueError),                                             # consistent, but on the CPU
    (dict(x=torch.zeros(N, H, dtype=torch.float64)), TypeError),
    (dict(x=torch.zeros(H)), ValueError),
    (dict(x=torch.zeros(N, 2, H)), ValueError),
    (dict(x=torch.zeros(N, 0), weight=None, bias=None), ValueError),
    (dict(x=torch.zeros(H, N).t()), ValueError),
    (dict(x=torch.zeros(1, H).expand(N, H)), ValueError),         # rows that overlap
    (dict(weight=torch.ones(H, dtype=torch.bfloat16)), TypeError),
    (dict(x=torch.zeros(N, H, dtype=torch.bfloat16), bias=torch.zeros(H, dtype=torch.bfloat16)), TypeError),
    (dict(weight=torch.ones(H + 1)), ValueError),
    (dict(weight=torch.ones(1, H)), ValueError),
    (dict(bias=torch.zeros(2 * H)[::2]), ValueError),
    (dict(eps=-1e-5), ValueError),
    (dict(eps=float("nan")), ValueError),
    (dict(eps=float("inf")), ValueError),
])
def test_layer_norm_rejects(change, exc):
    a = dict(x=torch.zeros(N, H), weight=torch.ones(H), bias=torch.zeros(H), eps=1e-5)
    a.update(change)
    with pytest.raises(exc):
        flce.layer_norm(a["x"], a["weight"], a["bias"], eps=a["eps"])


def _params(**kw):
    a = dict(rows=N, cols=H, ld_x=0, ld_grad=0, dtype=1, param_dtype=1, eps=1e-5, reserved=0)
    a.update(kw)
    return flce.flce_norm_params(*a.values())


def test_abi_codes():
    bad, odd = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED
    for change, code in ((dict(rows=-1), bad), (dict(cols=0), bad), (dict(ld_x=H - 1), bad), (dict(ld_grad=H - 1), bad),
                         (dict(ld_x=-H), bad), (dict(dtype=3), bad), (dict(dtype=-1), bad), (dict(param_dtype=2), bad),
                         (dict(eps=-1.0), bad), (dict(eps=float("nan")), bad), (dict(eps=float("inf")), bad),
                         (dict(reserved=1), bad), (dict(rows=(1 << 31) + 1), odd), (dict(cols=(1 << 20) + 1), odd),
                         (dict(rows=1 << 31, ld_x=1 << 20), odd), (dict(rows=1 << 31, ld_grad=1 << 62), odd)):
        p = _params(**change)
        with pytest.raises(flce.FlceError) as e:
            flce.flce_layer_norm_workspace_size(p)
        assert e.value.code == code, change
        assert flce.flce_layer_norm_forward(p, 16, 16, 16, 16, 16, 16, None) == code, change
        assert flce.flce_layer_norm_backward(p, 16, 16, 16, 16, 16, 16, 16, 16, 16, 1 << 40, None) == code, change
    p = _params()
    need = flce.flce_layer_norm_workspace_size(p)

    def fwd(x=16, w=16, b=16, y=16, m=16, r=16):
        return flce.flce_layer_norm_forward(p, x, w, b, y, m, r, None)

    def bwd(x=16, w=16, m=16, r=16, g=16, gx=16, gw=16, gb=16, ws=16, n=need):
        return flce.flce_layer_norm_backward(p, x, w, m, r, g, gx, gw, gb, ws, n, None)

    for name in ("x", "y", "m", "r"):
        assert fwd(**{name: None}) == bad, name
    for name in ("x", "w", "b", "y", "m", "r"):
        assert fwd(**{name: 17}) == odd, name
    for name in ("x", "m", "r", "g", "ws"):
        assert bwd(**{name: None}) == bad, name
    for name in ("x", "w", "m", "r", "g", "gx", "gw", "gb", "ws"):
        assert bwd(**{name: 17}) == odd, name
    assert bwd(n=need - 1) == flce.FLCE_ERR_WORKSPACE_TOO_SMALL


def test_definition_against_differences():
    """Central differences of the fp64 values: off by t^2 / 6 of the third derivative, here below 1e-8 (t = 1e-4
    and derivatives of order 10), and by 2^-52 of the sum over t, 1e-10."""
    rng = np.random.default_rng(1)
    x, w, b, g = rng.normal(size=(5, 9)), rng.normal(size=9), rng.normal(size=9), rng.normal(size=(5, 9))
    dx, dw, db = eo.layer_norm_grads(x, w, 1e-3, g)
    for k, grad in enumerate((dx, dw, db)):
        v = rng.normal(size=grad.shape)
        v /= np.abs(v).max()
        a, t = [x, w, b], 1e-4

        def f(s):
            moved = list(a)
            moved[k] = a[k] + s * v
            return (g * eo.layer_norm(*moved, 1e-3)[0]).sum()

        assert abs((f(t) - f(-t)) / (2 * t) - (grad * v).sum()) < 1e-6
