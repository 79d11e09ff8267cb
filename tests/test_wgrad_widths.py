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


@pytest.mark.parametrize("width", [1 << 26, (1 << 26) + 8, 1 << 30])
def test_slices_of_rows_past_32_bit_offsets_are_refused(lib, width):
    """32 rows of 2^26 bf16 columns are 2^32 bytes: their range, taken in 32 bits, would be empty, and the products 0."""
    w = lib.moe_grouped_gemm_wgrad
    assert w(FAKE, FAKE, FAKE, 1, 64, width, 8, FAKE, None) == _lib.MOE_ERR_UNSUPPORTED
    assert w(FAKE, FAKE, FAKE, 1, 64, 8, width, FAKE, None) == _lib.MOE_ERR_UNSUPPORTED
    assert lib.moe_grouped_gemm_wgrad_grid(FAKE, FAKE, FAKE, 1, 1, 8, width, FAKE, 8, None) == _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.gpu
def test_the_widest_slices_that_are_taken():
    """Just below: 40 rows of 2^26 - 8 columns, a k-slice and a part of one, against exact small integers."""
    import torch

    import mixture_experts_ffn_group_amd as moe
    dev = "cuda:0"
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info(dev)[0] < 60 << 30:
        pytest.skip("needs 30 GB of device memory")
    M, W = 40, (1 << 26) - 8
    ids = torch.arange(W, dtype=torch.int32, device=dev)
    wide = torch.empty((M, W), dtype=torch.bfloat16, device=dev)
    for r in range(M):
        wide[r] = ((ids + 3 * r) % 7 - 3).to(torch.bfloat16)
    narrow = torch.randint(-2, 3, (M, 8), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(dev)
    off = torch.tensor([0, 37], dtype=torch.int32, device=dev)  # sums of at most 37 * 6: whole bf16 numbers below 256
    period = wide[:37, :7].float().t() @ narrow[:37].float()
    ref = period.to(torch.bfloat16)[(ids % 7).long()]
    assert torch.equal(moe.grouped_gemm_wgrad(wide, narrow, off, 1)[0], ref)
    assert torch.equal(moe.grouped_gemm_wgrad(narrow, wide, off, 1)[0], ref.t())
    del wide, ref, ids
    torch.cuda.empty_cache()
