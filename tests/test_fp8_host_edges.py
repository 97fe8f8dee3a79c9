"""Host side of the block-scaled E4M3 and scored-router entry points at the edges of their arguments (no GPU)."""
import ctypes

import pytest
import torch

import nvfp4_weight_only_top_b200 as moe
from nvfp4_weight_only_top_b200 import _abi

BAD, UNS = _abi.ERR_INVALID_ARG, _abi.ERR_UNSUPPORTED
A, B = 0x20000, 0x40000            # aligned addresses, never read


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _passes_the_checks(rc):
    """True where only the device is missing (or, with one, nothing is)."""
    return rc == _abi.OK if torch.cuda.is_available() else rc == UNS and "no CUDA device" in moe.moe_nvfp4_last_error()


def test_quantize_no_rows_into_expert_order():
    """An empty tensor's address is NULL: inv is then not there, and k is still the router's."""
    quantize = moe.lib().moe_nvfp4_fp8_quantize
    assert torch.empty(0, dtype=torch.int32).data_ptr() == 0
    for k in (1, 4, 32):
        assert _passes_the_checks(quantize(None, 0, 256, None, k, None, None, None)), k
    for k in (0, 33):
        assert quantize(None, 0, 256, None, k, None, None, None) == BAD
    assert quantize(_p(A), 1, 256, None, 4, _p(B), _p(B), None) == BAD
