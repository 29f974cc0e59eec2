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
