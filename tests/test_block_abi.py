"""The calls around the layer on the CPU: declared, bound, and refused on the host without a handle."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.load_builder().build()
    import mixture_experts_layer_48_b200 as m
    return m


NAMES = ("moe_grouped_matmul", "moe_grouped_wgrad", "moe_swiglu", "moe_swiglu_backward", "moe_block_norm",
         "moe_block_norm_workspace_bytes", "moe_block_norm_backward")


def test_calls_are_bound(lib):
    for name in NAMES:
        assert name in lib.EXPORTED
    for name in ("grouped_matmul", "grouped_wgrad", "swiglu", "swiglu_backward", "block_norm", "block_norm_backward",
                 "block_norm_workspace_bytes", "block"):
        assert callable(getattr(lib.Moe, name))


@pytest.mark.parametrize("name", [n for n in NAMES if not n.endswith("_bytes")])
def test_null_handle_is_refused(lib, name):
    f = getattr(lib, name)
    zero = {ctypes.c_int: 0, ctypes.c_float: 1.0, ctypes.c_size_t: 0, ctypes.c_void_p: None}
    assert f(*[zero[t] for t in f.argtypes]) == lib.MOE_ERR_ARG
    one = dict(zero)
    one[ctypes.c_int] = 8
    assert f(*[one[t] for t in f.argtypes]) == lib.MOE_ERR_ARG


def test_workspace_of_a_null_handle(lib):
    assert lib.moe_block_norm_workspace_bytes(None, 16) == 0


def test_dtype_codes(lib):
    import torch
    assert lib._dtype(torch.bfloat16, "x") == lib.MOE_BF16 == 0
    assert lib._dtype(torch.float32, "x") == lib.MOE_F32 == 1
    for bad in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError):
            lib._dtype(bad, "x")
