"""Sizes the library takes in 32 bits: ctypes keeps the low 32 bits of a larger number, so the binding has to refuse
it, or 2^32 + 2 picks would be 2."""
import pytest
import torch

import mixture_experts_ffn_group_amd as moe
from mixture_experts_ffn_group_amd import _lib

DEV = "cuda:0"
B = 1 << 32


@pytest.mark.parametrize("i", [1, 2, 3, 4])
@pytest.mark.parametrize("v", [B + 64, B // 2, -B + 64])
def test_layer_shapes(i, v):
    sizes = [1, 64, 64, 8, 2]
    sizes[i] = v
    with pytest.raises(ValueError, match="32 bits"):
        _lib.shape(*sizes)
    with pytest.raises(ValueError, match="32 bits"):
        moe.query_support(*sizes)


def test_shapes_that_fit_go_to_the_library():
    assert _lib.shape(B, B // 2 - 1, 64, 8, 2).emb == B // 2 - 1  # T has 64 bits
    assert _lib.shape(1, 64, 64, 8, -B // 2).k == -B // 2
    for k in (0, -1, 9):
        with pytest.raises(moe.MoeError):
            moe.query_support(1, 64, 64, 8, k)


@pytest.mark.parametrize("i", [0, 1, 2])
@pytest.mark.parametrize("v", [B + 1, -B + 1])
def test_router_sizes(i, v):
    groups = [1, 1, 1]
    groups[i] = v
    with pytest.raises(ValueError, match="32 bits"):
        moe._router("softmax", *groups, True, 1.0)


@pytest.mark.parametrize("kw", [dict(N=B + 256), dict(Q=B + 256), dict(grid=B + 8)])
def test_tile_schedule_sizes(kw):
    with pytest.raises(ValueError, match="32 bits"):
        moe.tile_schedule("wgrad", [0, 5, 9], **dict(dict(M=9, N=256, grid=8, Q=256), **kw))


@pytest.mark.gpu
def test_calls_refuse_them_before_they_allocate():
    l = torch.zeros((2, 8), device=DEV)
    c, s = moe.ckpt_quantize(torch.zeros((4, 64), device=DEV))
    D = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    slot = torch.arange(4, dtype=torch.int32, device=DEV)
    w = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: moe.route_scored(B + 2, l), lambda: moe.route_scored(2, l, n_group=B + 4, topk_group=2),
                 lambda: moe.ckpt_dequantize(c, s, slot, B + 2), lambda: moe.mx_quantize_rows(D, slot, B + 2),
                 lambda: moe.grouped_gemm_wgrad_ckpt(c, s, D, off, 2, slot, B + 1),
                 lambda: moe.grouped_gemm(D, w, off, row_slot=slot, slot_div=B + 1),
                 lambda: moe.grouped_gemm_wgrad(D, D, off, 2, grid=B + 8)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


@pytest.mark.gpu
def test_rows_longer_than_32_bits():
    """Tensors whose row length the library would have taken as 32."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info(DEV)[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.empty((1, B + 32), dtype=torch.bfloat16, device=DEV)
    codes = torch.empty((1, B + 32), dtype=torch.int8, device=DEV)
    scales = torch.empty((1, B // 32 + 1), dtype=torch.uint8, device=DEV)
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    held = torch.cuda.memory_allocated(DEV)
    for call in (lambda: moe.ckpt_quantize(x), lambda: moe.ckpt_dequantize(codes, scales),
                 lambda: moe.swiglu_bwd_ckpt(x, codes, scales),
                 lambda: moe.grouped_gemm_wgrad_ckpt(codes, scales, x, off, 1), lambda: moe.mx_quantize_rows(x)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
        assert torch.cuda.memory_allocated(DEV) == held
    del x, codes, scales
    torch.cuda.empty_cache()
