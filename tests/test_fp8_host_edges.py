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


def _matmul():
    return moe.lib().moe_nvfp4_fp8_matmul(_p(A), _p(A), 0, _p(B), _p(B), 1, 128, 256, None, _p(B), 0, None)


@pytest.mark.parametrize("tile", ["64", "128", "256", "64x1", "64x8", "128x2", ""])
def test_forced_tiles(tile, monkeypatch):
    monkeypatch.setenv("MOE_NVFP4_FP8_TILE", tile)
    assert _passes_the_checks(_matmul())


@pytest.mark.parametrize("tile", ["wide", "32", "640", "64x", "64x0", "64x9", "64x10", "256x2", "64 ", " 64", "128X2", "-64"])
def test_unreadable_tiles_are_refused(tile, monkeypatch):
    """Not taken for one of the tiles."""
    monkeypatch.setenv("MOE_NVFP4_FP8_TILE", tile)
    assert _matmul() == BAD
    assert "MOE_NVFP4_FP8_TILE" in moe.moe_nvfp4_last_error()


WIDE = (1 << 32) + 256             # 256 where only 32 bits are kept


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda: moe.moe_nvfp4_route(_meta(1, WIDE, dtype=torch.float32), 4),
    lambda: moe.moe_nvfp4_route_scored(_meta(1, WIDE, dtype=torch.float32), moe.make_router(), 4),
    lambda: moe.moe_nvfp4_fp8_quantize(_meta(1, WIDE)),
    lambda: moe.moe_nvfp4_fp8_quantize(_meta(1, 256), inv=_meta(4, dtype=torch.int32), k=(1 << 32) + 4),
    lambda: moe.moe_nvfp4_fp8_swiglu_quantize(_meta(1, 2 * WIDE)),
    lambda: moe.moe_nvfp4_fp8_quantize_weights(_meta(2, WIDE, 256)),
    lambda: moe.moe_nvfp4_fp8_quantize_weights(_meta(256, WIDE)),
    lambda: moe.moe_nvfp4_fp8_matmul(_meta(1, WIDE), None, _meta(256, WIDE), None),
    lambda: moe.moe_nvfp4_fp8_matmul(_meta(1, 256), None, _meta(WIDE, 256), None),
    lambda: moe.moe_nvfp4_fp8_matmul(_meta(1, 256), None, _meta(WIDE, 8, 256), None, _meta(1, dtype=torch.int32)),
    lambda: moe.moe_nvfp4_gather_rows(_meta(1, WIDE), _meta(2, dtype=torch.int32), 2),
    lambda: moe.moe_nvfp4_combine(_meta(2, WIDE, dtype=torch.float32), _meta(1, 2, dtype=torch.float32), None, 2),
    lambda: moe.moe_nvfp4_encode(_meta(1, WIDE, 256), _meta(16, dtype=torch.uint8), 0, 0, 0, 0),
    lambda: moe.make_router(groups=(1 << 32) + 8),
    lambda: moe.make_router(groups=8, top_groups=(1 << 32) + 4),
    lambda: moe.make_router(groups=8, group_top=(1 << 32) + 2),
])
def test_sizes_past_32_bits_are_refused(call):
    """Not taken modulo 2^32."""
    with pytest.raises(ValueError, match="32 bits"):
        call()


def _route(T, k, E=64):
    r = moe.make_router()
    return moe.lib().moe_nvfp4_route_scored(_p(A), T, E, ctypes.byref(r), k, *[_p(B)] * 6, None)


def test_routed_rows_fit_32_bits():
    """2^26 tokens of 32 choices are 2^31 rows, one more than the last offset can say."""
    for T, k in ((1 << 26, 32), ((1 << 26) + 1, 1)):
        assert _route(T, k) == UNS and "too large" in moe.moe_nvfp4_last_error()
        assert moe.lib().moe_nvfp4_route(_p(A), T, 64, k, *[_p(B)] * 6, None) == UNS
        assert "too large" in moe.moe_nvfp4_last_error()
    if not torch.cuda.is_available():
        for T, k in (((1 << 26) - 1, 32), (1 << 26, 31)):
            assert _passes_the_checks(_route(T, k))


@pytest.mark.parametrize("which", range(7))
def test_misaligned_router_pointers_are_refused(which):
    ptrs = [A] + [B] * 6
    ptrs[which] += 2
    r = moe.make_router()
    rc = moe.lib().moe_nvfp4_route_scored(_p(ptrs[0]), 4, 64, ctypes.byref(r), 4, *[_p(v) for v in ptrs[1:]], None)
    assert rc == BAD and "aligned" in moe.moe_nvfp4_last_error()
