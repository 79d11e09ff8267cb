"""Widths of the weight gradients at the ends of their 32-bit arithmetic: refused before anything is enqueued."""
import ctypes as C

import pytest

from mixture_experts_ffn_group_amd import _lib

FAKE = C.c_void_p(0x1000)  # never dereferenced
TOP = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


@pytest.mark.parametrize("below", [8, 32, 96, 104, 128, 224, 248])
def test_tile_counts_do_not_overflow(lib, below):
    P = TOP - below
    assert lib.moe_grouped_gemm_wgrad(FAKE, FAKE, FAKE, 1, 1, P, 8, FAKE, None) == _lib.MOE_ERR_UNSUPPORTED
    assert lib.moe_grouped_gemm_wgrad(FAKE, FAKE, FAKE, 1, 1, 8, P, FAKE, None) == _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("below", [32, 64, 96])
def test_tile_counts_from_checkpoints_do_not_overflow(lib, below):
    P = TOP - below
    assert lib.moe_grouped_gemm_wgrad_ckpt(FAKE, FAKE, 1, FAKE, 1, FAKE, FAKE, 1, 64, P, 8, FAKE, None, 0, None) == \
        _lib.MOE_ERR_UNSUPPORTED
    assert lib.moe_wgrad_ckpt_workspace_bytes(1, 1 << 16, P, 8) == 0
    widest = lib.moe_wgrad_ckpt_workspace_bytes(1, 1 << 16, TOP - 128, 8)
    assert 0 < widest < 1 << 40
