"""embedding, embedding_backward and their C entry points refuse what the kernels cannot take (CPU only)."""
import pytest
import torch

import linear_cross_entropy_tiled_amd as flce

N, H, V = 6, 8, 20
IDS = torch.zeros(N, dtype=torch.int64)


@pytest.mark.parametrize("change,exc", [
    ({}, ValueError),                                             # consistent, but on the CPU
    (dict(ids=torch.zeros(N)), TypeError),
    (dict(ids=torch.zeros(2, 3, dtype=torch.int64)), ValueError),
    (dict(ids=torch.zeros(2 * N, dtype=torch.int32)[::2]), ValueError),
    (dict(weight=torch.zeros(V, H, dtype=torch.float64)), TypeError),
    (dict(weight=torch.zeros(V)), ValueError),
    (dict(weight=torch.zeros(0, H)), ValueError),
    (dict(weight=torch.zeros(V, 0)), ValueError),
    (dict(weight=torch.zeros(H, V).t()), ValueError),
    (dict(scale=float("inf")), ValueError),
    (dict(scale=float("nan")), ValueError),
])
def test_embedding_rejects(change, exc):
    a = dict(ids=IDS, weight=torch.zeros(V, H), scale=1.0)
    a.update(change)
    with pytest.raises(exc):
        flce.embedding(a["ids"], a["weight"], scale=a["scale"])


@pytest.mark.parametrize("change,exc", [
    ({}, ValueError),
    (dict(ids=torch.zeros(N + 1, dtype=torch.int64)), ValueError),
    (dict(grad=torch.zeros(N)), ValueError),
    (dict(grad=torch.zeros(N, 0)), ValueError),
    (dict(grad=torch.zeros(N, H, dtype=torch.int8)), TypeError),
    (dict(grad=torch.zeros(H, N).t()), ValueError),
    (dict(vocab=0), ValueError),
    (dict(scale=float("inf")), ValueError),
    (dict(grad_weight=torch.zeros(V, H + 1)), ValueError),
    (dict(grad_weight=torch.zeros(V + 1, H)), ValueError),
    (dict(grad_weight=torch.zeros(H, V).t()), ValueError),
    (dict(grad_weight=torch.zeros(V, H, dtype=torch.float64)), TypeError),
    (dict(grad_weight_dtype="f64"), ValueError),
])
def test_embedding_backward_rejects(change, exc):
    a = dict(grad=torch.zeros(N, H), ids=IDS, vocab=V)
    a.update(change)
    with pytest.raises(exc):
        flce.embedding_backward(**a)


def _params(**kw):
    a = dict(n=N, h=H, v=V, ignore=-100, dtype=1, gdtype=0, flags=0, scale=1.0)
    a.update(kw)
    return flce.flce_embedding_params(*a.values())


def test_abi_codes():
    bad, odd = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED
    for change, code in ((dict(n=-1), bad), (dict(h=0), bad), (dict(v=0), bad), (dict(dtype=3), bad), (dict(gdtype=-1), bad),
                         (dict(flags=2), bad), (dict(flags=8), bad), (dict(scale=float("nan")), bad),
                         (dict(n=1 << 31), odd), (dict(v=1 << 31), odd), (dict(h=(1 << 20) + 1), odd),
                         (dict(n=(1 << 31) - 1, h=1 << 20), odd), (dict(v=(1 << 31) - 1, h=1 << 10), odd)):
        p = _params(**change)
        with pytest.raises(flce.FlceError) as e:
            flce.flce_embedding_workspace_size(p)
        assert e.value.code == code, change
        assert flce.flce_embedding_forward(p, 16, 16, 16, None) == code, change
        assert flce.flce_embedding_backward(p, 16, 16, 16, 16, 1 << 50, None) == code, change
    for flags, ids_bad in ((0, 20), (4, 18)):
        p = _params(flags=flags)
        need = flce.flce_embedding_workspace_size(p)

        def fwd(ids=16, w=16, out=16):
            return flce.flce_embedding_forward(p, ids, w, out, None)

        def bwd(ids=16, g=16, gw=16, ws=16, n=need):
            return flce.flce_embedding_backward(p, ids, g, gw, ws, n, None)

        for name in ("ids", "w", "out"):
            assert fwd(**{name: None}) == bad, name
        for name in ("ids", "g", "gw", "ws"):
            assert bwd(**{name: None}) == bad, name
        assert fwd(ids=ids_bad) == bwd(ids=ids_bad) == odd
        for name in ("w", "out"):
            assert fwd(**{name: 17}) == odd, name
        assert bwd(g=17) == bwd(gw=18) == bwd(ws=24) == odd
        assert bwd(n=need - 1) == flce.FLCE_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("n", [0, 1, 31, 8192, 8193, 131073, 5_000_000, (1 << 31) - 1])
def test_workspace_holds_the_sorts_buffers(n):
    need = flce.flce_embedding_workspace_size(_params(n=n, h=1))
    pairs = 1 if n <= 16384 else 2                    # of a key and a token number
    assert 8 * pairs * n <= need <= 8 * pairs * n + (1 << 20) + n
