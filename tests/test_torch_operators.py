"""The operators of libflce_torch.so as a recorded graph calls them: their arguments say everything themselves."""
import os

import pytest

import linear_cross_entropy_tiled_amd as flce

OPERATORS = ("_layer_norm", "_embedding", "_quantize_mxfp4", "_dequantize_mxfp4", "_logprobs_mxfp4")


@pytest.fixture(scope="module")
def ops():
    if not os.path.exists(flce.TORCH_LIB_PATH):
        pytest.skip("libflce_torch.so is not built")
    return flce.torch_ops()


@pytest.mark.parametrize("name", OPERATORS)
def test_no_argument_is_an_address(ops, name):
    """A trace keeps an operator's numbers as constants: whole numbers are sizes or ids, never what a pointer was."""
    whole = [a.name for a in getattr(ops, name).default._schema.arguments if str(a.type) == "int"]
    assert set(whole) <= {"workspace", "ignore_index", "dtype"}, whole


def _norm(**kw):
    import torch
    a = dict(x=torch.zeros(4, 64), weight=torch.ones(64), bias=torch.zeros(64), eps=1e-5, workspace=1 << 20)
    return {**a, **kw}


def _embedding(**kw):
    import torch
    a = dict(ids=torch.zeros(4, dtype=torch.int64), weight=torch.ones(10, 64), scale=1.0, ignore_index=-100,
             workspace=1 << 20)
    return {**a, **kw}


def _scores(**kw):
    import torch
    u8 = torch.uint8
    a = dict(hidden=torch.zeros(4, 64), hidden_scale=None, weight=torch.zeros(10, 32, dtype=u8),
             weight_scale=torch.zeros(10, 2, dtype=u8), bias=torch.zeros(10), targets=torch.zeros(4, dtype=torch.int64),
             logit_scale=1.0, softcap=0.0, ignore_index=-100, workspace=1 << 20, entropy=False)
    return {**a, **kw}


def _cases():
    import torch
    z, u8 = torch.zeros, torch.uint8
    for kw in (dict(x=z(4, 128)), dict(x=z(64)), dict(x=z(4, 64).double()), dict(x=z(64, 4).t()), dict(weight=z(63)),
               dict(bias=z(1, 64)), dict(weight=z(128)[::2]), dict(bias=z(64).half()), dict(weight=None, bias=z(65)), {}):
        yield "_layer_norm", _norm(**kw)
    for kw in (dict(ids=z(2, 2, dtype=torch.int64)), dict(ids=z(4)), dict(ids=z(8, dtype=torch.int64)[::2]),
               dict(weight=z(64)), dict(weight=z(10, 128)[:, ::2]), dict(weight=z(10, 64).double()), dict(weight=z(0, 64)),
               {}):
        yield "_embedding", _embedding(**kw)
    for x in (z(4, 48), z(4, 0), z(32), z(4, 64).double(), z(4, 128)[:, ::2], z(4, 64)):
        yield "_quantize_mxfp4", dict(x=x)
    q, s = z(4, 32, dtype=u8), z(4, 2, dtype=u8)
    for a in ((q, s[:3], torch.float32), (q, z(4, 3, dtype=u8), torch.float32), (q.int(), s, torch.float32),
              (q, s.int(), torch.float32), (q, s, torch.float64), (z(4, 24, dtype=u8), s, torch.float32),
              (q, s, torch.float32)):
        yield "_dequantize_mxfp4", dict(zip(("q", "scale", "dtype"), a))
    for kw in (dict(hidden=z(4, 96)), dict(hidden=z(5, 64)), dict(hidden=z(4, 64).double()), dict(hidden=z(4, 32, dtype=u8)),
               dict(hidden=z(4, 32, dtype=u8), hidden_scale=z(4, 3, dtype=u8)), dict(hidden_scale=z(4, 2, dtype=u8)),
               dict(hidden=z(4, 16, dtype=u8), hidden_scale=z(4, 1, dtype=u8)), dict(weight=z(11, 32, dtype=u8)),
               dict(weight_scale=z(10, 2)), dict(bias=z(9)), dict(bias=z(10).half()), dict(targets=z(3, dtype=torch.int64)),
               dict(targets=z(4)), dict(targets=z(8, dtype=torch.int64)[::2]), {}):
        yield "_logprobs_mxfp4", _scores(**kw)


@pytest.mark.parametrize("name", OPERATORS)
def test_tensors_that_the_kernels_cannot_take_are_refused(ops, name):
    """Also without the Python function in front, as a recorded graph calls them with other tensors than it was recorded
    with.  (The last case of each is refused for its device alone.)"""
    cases = [kw for op, kw in _cases() if op == name]
    assert len(cases) >= 6
    for kw in cases:
        with pytest.raises(RuntimeError, match="type, size, layout or device"):
            getattr(ops, name)(**kw)
