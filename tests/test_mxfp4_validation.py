"""quantize_mxfp4, dequantize_mxfp4, token_logprobs_mxfp4 and their C entry points refuse what the kernels cannot
take; the oracle's MXFP4 against the format's own properties (CPU only)."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_tiled_amd as flce
from oracle import mx_oracle as mo

N, H, V = 16, 64, 100
U8 = torch.uint8


def _args(**kw):
    a = dict(hidden=torch.zeros(N, H), weight=torch.zeros(V, H // 2, dtype=U8), weight_scale=torch.zeros(V, H // 32, dtype=U8),
             targets=torch.zeros(N, dtype=torch.int64), bias=None, hidden_scale=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("change,exc", [
    ({}, ValueError),                                                          # consistent, but on the CPU
    (dict(weight=torch.zeros(V, H // 2, dtype=torch.int8)), TypeError),
    (dict(weight=torch.zeros(V, H // 2 + 16, dtype=U8)), ValueError),
    (dict(weight=torch.zeros(V, H // 2 + 16, dtype=U8), weight_scale=torch.zeros(V, 3, dtype=U8)), ValueError),
    (dict(weight=torch.zeros(V, 24, dtype=U8)), ValueError),
    (dict(weight=torch.zeros(V, 0, dtype=U8), weight_scale=torch.zeros(V, 0, dtype=U8), hidden=torch.zeros(N, 0)), ValueError),
    (dict(weight=torch.zeros(V * H, dtype=U8)), ValueError),
    (dict(weight_scale=torch.zeros(V, H // 32)), TypeError),
    (dict(weight_scale=torch.zeros(V, H // 32 + 1, dtype=U8)), ValueError),
    (dict(weight_scale=torch.zeros(V - 1, H // 32, dtype=U8)), ValueError),
    (dict(hidden=torch.zeros(N, H // 2, dtype=U8)), TypeError),                # without its scale
    (dict(hidden_scale=torch.zeros(N, H // 32, dtype=U8)), TypeError),         # a scale for unquantized states
    (dict(hidden=torch.zeros(N, H // 2, dtype=U8), hidden_scale=torch.zeros(N, 1, dtype=U8)), ValueError),
    (dict(hidden=torch.zeros(N, H, dtype=torch.float64)), TypeError),
    (dict(hidden=torch.zeros(H, N).t()), ValueError),
    (dict(hidden=torch.zeros(N * H)), ValueError),
    (dict(weight=torch.zeros(H // 2, V, dtype=U8).t()), ValueError),
    (dict(bias=torch.zeros(V, dtype=torch.bfloat16)), TypeError),
    (dict(bias=torch.zeros(V + 1)), ValueError),
    (dict(targets=torch.zeros(N)), TypeError),
    (dict(targets=torch.zeros(N - 1, dtype=torch.int64)), ValueError),
])
def test_token_logprobs_mxfp4_rejects(change, exc):
    a = _args(**change)
    with pytest.raises(exc):
        flce.token_logprobs_mxfp4(a["hidden"], a["weight"], a["weight_scale"], a["targets"], a["bias"],
                                  hidden_scale=a["hidden_scale"])


@pytest.mark.parametrize("x,exc", [
    (torch.zeros(4, 32), ValueError), (torch.zeros(4, 48), ValueError), (torch.zeros(4, 0), ValueError),
    (torch.zeros(64), ValueError), (torch.zeros(32, 32).t(), ValueError), (torch.zeros(4, 32, dtype=U8), TypeError)])
def test_quantize_mxfp4_rejects(x, exc):
    with pytest.raises(exc):
        flce.quantize_mxfp4(x)


@pytest.mark.parametrize("q,s,dtype,exc", [
    (torch.zeros(4, 16, dtype=U8), torch.zeros(4, 1, dtype=U8), None, ValueError),
    (torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 1, dtype=U8), None, TypeError),
    (torch.zeros(4, 16, dtype=U8), torch.zeros(4, 1), None, TypeError),
    (torch.zeros(4, 24, dtype=U8), torch.zeros(4, 1, dtype=U8), None, ValueError),
    (torch.zeros(4, 16, dtype=U8), torch.zeros(4, 2, dtype=U8), None, ValueError),
    (torch.zeros(4, 16, dtype=U8), torch.zeros(3, 1, dtype=U8), None, ValueError),
    (torch.zeros(64, dtype=U8), torch.zeros(4, 1, dtype=U8), None, ValueError),
    (torch.zeros(4, 16, dtype=U8), torch.zeros(4, 1, dtype=U8), torch.float64, TypeError),
    (torch.zeros(16, 16, dtype=U8).t(), torch.zeros(16, 1, dtype=U8), None, ValueError)])
def test_dequantize_mxfp4_rejects(q, s, dtype, exc):
    with pytest.raises(exc):
        flce.dequantize_mxfp4(q, s, dtype)


def test_abi_codes():
    bad, odd = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED
    for a, code in (((3, 16, 4, 32, 16, 16), bad), ((1, 16, -1, 32, 16, 16), bad), ((1, 16, 4, 0, 16, 16), bad),
                    ((1, None, 4, 32, 16, 16), bad), ((1, 16, 4, 32, None, 16), bad), ((1, 16, 4, 32, 16, None), bad),
                    ((1, 16, 4, 48, 16, 16), odd), ((1, 24, 4, 32, 16, 16), odd), ((1, 16, 4, 32, 24, 16), odd),
                    ((1, 16, 1 << 31, 32, 16, 16), odd), ((1, 16, 4, 1 << 31, 16, 16), odd)):
        assert flce.flce_quantize_mxfp4(*a, None) == code, a
        d, x, r, c, q, s = a
        assert flce.flce_dequantize_mxfp4(d, q, s, r, c, x, None) == code, a
    for opts, code in ((dict(reduction="sum"), bad), (dict(z_loss=0.1), bad), (dict(h=48), odd), (dict(h=0), bad),
                       (dict(h=(1 << 18) + 32), odd), (dict(n=1 << 26, h=64), odd)):
        n, h = opts.pop("n", N), opts.pop("h", H)
        p = flce.make_params(n, h, V, **{"reduction": "none", **opts})
        with pytest.raises(flce.FlceError) as e:
            flce.flce_logprobs_mxfp4_workspace_size(p)
        assert e.value.code == code
        assert flce.flce_logprobs_mxfp4(p, 16, 16, 16, 16, None, 16, 16, None, 16, 16, 1 << 40, None) == code
    p = flce.make_params(N, H, V, reduction="none")
    need = flce.flce_logprobs_mxfp4_workspace_size(p)

    def call(x=16, s=16, w=16, ws=16, b=None, t=16, lp=16, lse=16, work=16, n=need):
        return flce.flce_logprobs_mxfp4(p, x, s, w, ws, b, t, lp, None, lse, work, n, None)

    for name in ("x", "w", "ws", "t", "lp", "lse", "work"):    # (without s, x holds values)
        assert call(**{name: None}) == bad, name
    for name in ("x", "w", "b", "work"):
        assert call(**{name: 24}) == odd, name
    assert call(s=18) == odd and call(ws=18) == odd and call(t=20) == odd and call(lp=18) == odd
    assert call(n=need - 1) == flce.FLCE_ERR_WORKSPACE_TOO_SMALL


def test_the_oracles_format():
    """Values of the grid keep themselves, ties go to the even code, a value never moves past its neighbours, scales
    are the specification's."""
    assert mo.quantize(np.concatenate([mo.GRID] * 4)[None])[1][0, 0] == 127
    code, s = mo.quantize(np.concatenate([mo.GRID, -mo.GRID, mo.GRID, -mo.GRID])[None] * 8)
    assert s[0, 0] == 130 and np.array_equal(code[0, :16], np.arange(16))
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9])
    code, s = mo.quantize(np.concatenate([mids] * 4)[None])
    assert s[0, 0] == 127 and code[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    x = np.random.default_rng(0).normal(size=(20, 96)).astype(np.float32)
    v = mo.values(*mo.quantize(x))
    unit = np.repeat(np.exp2(mo.quantize(x)[1].astype(float) - 127), 32, axis=1)
    assert np.all(np.abs(v - x)[np.abs(x) <= 6 * unit] <= (unit * 1.0)[np.abs(x) <= 6 * unit])
    assert np.array_equal(mo.values(*mo.quantize(v)), v)
    assert np.array_equal(mo.unpack(mo.pack(code)), code)
