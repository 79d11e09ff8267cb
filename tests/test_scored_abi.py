"""Refusals of the score router and of the 8-bit checkpoint calls: host validation, no GPU, nothing enqueued."""
import ctypes as C
import os

import pytest
import torch

import mixture_experts_ffn_group_amd as moe
from mixture_experts_ffn_group_amd import _lib

FAKE, ODD = C.c_void_p(0x1000), C.c_void_p(0x1001)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_ffn_group_amd import build
        build.build()
    return _lib.lib()


def _router(score=1, n_group=4, topk_group=2, group_top=2, renorm=1, scale=1.0):
    return _lib.MoeRouter(score, n_group, topk_group, group_top, renorm, scale)


@pytest.mark.parametrize("kw", [dict(score=2), dict(n_group=0), dict(n_group=3), dict(topk_group=0),
                                dict(topk_group=5), dict(group_top=0), dict(group_top=3), dict(n_group=16),
                                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                                dict(scale=float("nan")), dict(topk_group=1)])
def test_router_refusals(lib, kw):
    s = _lib.shape(8, 64, 64, 16, 5)  # groups of four: topk_group=1 leaves fewer than k experts
    r = _router(**kw)
    for call in (lambda: lib.moe_route_scored(C.byref(s), C.byref(r), FAKE, 0, None, FAKE, FAKE, None),
                 lambda: lib.moe_route_scored_bwd(C.byref(s), C.byref(r), FAKE, 0, FAKE, FAKE, FAKE, FAKE, None)):
        assert call() == _lib.MOE_ERR_SHAPE
        assert lib.moe_last_error_detail()


def test_route_scored_argument_refusals(lib):
    s, r = _lib.shape(8, 64, 64, 16, 5), _router()
    S, R = C.byref(s), C.byref(r)
    assert lib.moe_route_scored(None, R, FAKE, 0, None, FAKE, FAKE, None) == _lib.MOE_ERR_NULL
    assert lib.moe_route_scored(S, None, FAKE, 0, None, FAKE, FAKE, None) == _lib.MOE_ERR_NULL
    assert lib.moe_route_scored(S, R, FAKE, 7, None, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert lib.moe_route_scored(S, R, None, 0, None, FAKE, FAKE, None) == _lib.MOE_ERR_NULL
    assert lib.moe_route_scored(S, R, FAKE, 0, ODD, FAKE, FAKE, None) == _lib.MOE_ERR_ALIGN
    assert lib.moe_route_scored(S, R, FAKE, 0, None, FAKE, None, None) == _lib.MOE_ERR_NULL
    assert lib.moe_route_scored_bwd(S, R, FAKE, 0, FAKE, FAKE, None, FAKE, None) == _lib.MOE_ERR_NULL
    assert lib.moe_route_scored_bwd(S, R, FAKE, 0, FAKE, FAKE, FAKE, ODD, None) == _lib.MOE_ERR_ALIGN
    big = _lib.shape(8, 64, 64, 300, 5)
    assert lib.moe_route_scored(C.byref(big), R, FAKE, 0, None, FAKE, FAKE, None) == _lib.MOE_ERR_UNSUPPORTED
    none = _lib.shape(0, 64, 64, 16, 5)
    assert lib.moe_route_scored(C.byref(none), R, None, 0, None, None, None, None) == _lib.MOE_OK
    assert lib.moe_route_scored_bwd(C.byref(none), R, None, 0, None, None, None, None, None) == _lib.MOE_OK


def test_ckpt_refusals(lib):
    q, d, b = lib.moe_ckpt_quantize, lib.moe_ckpt_dequantize, lib.moe_swiglu_bwd_ckpt
    assert q(FAKE, 0, 4, 48, FAKE, FAKE, None) == _lib.MOE_ERR_UNSUPPORTED
    assert q(FAKE, 0, 4, 0, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(FAKE, 0, -1, 64, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(FAKE, 2, 4, 64, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(FAKE, 0, 1 << 40, 64, FAKE, FAKE, None) == _lib.MOE_ERR_UNSUPPORTED
    assert q(None, 0, 4, 64, FAKE, FAKE, None) == _lib.MOE_ERR_NULL
    assert q(FAKE, 0, 4, 64, ODD, FAKE, None) == _lib.MOE_ERR_ALIGN
    assert q(None, 1, 0, 64, None, None, None) == _lib.MOE_OK
    assert d(FAKE, FAKE, 4, 64, FAKE, 0, 8, FAKE, 0, None) == _lib.MOE_ERR_SHAPE
    assert d(FAKE, FAKE, 4, 64, None, 1, 8, FAKE, 0, None) == _lib.MOE_ERR_SHAPE
    assert d(FAKE, FAKE, 0, 64, FAKE, 1, 8, FAKE, 0, None) == _lib.MOE_ERR_SHAPE
    assert d(FAKE, FAKE, 4, 64, FAKE, 1, 8, FAKE, 5, None) == _lib.MOE_ERR_SHAPE
    assert d(FAKE, None, 4, 64, FAKE, 1, 8, FAKE, 1, None) == _lib.MOE_ERR_NULL
    assert d(None, None, 4, 64, None, 1, 0, None, 1, None) == _lib.MOE_OK
    assert b(4, 48, FAKE, FAKE, FAKE, None, None, FAKE, None, None, None) == _lib.MOE_ERR_UNSUPPORTED
    assert b(1 << 31, 64, FAKE, FAKE, FAKE, None, None, FAKE, None, None, None) == _lib.MOE_ERR_UNSUPPORTED
    assert b(4, 64, FAKE, FAKE, None, None, None, FAKE, None, None, None) == _lib.MOE_ERR_NULL
    assert b(4, 64, FAKE, FAKE, FAKE, None, ODD, FAKE, None, None, None) == _lib.MOE_ERR_ALIGN
    assert b(4, 64, FAKE, FAKE, FAKE, None, None, None, None, None, None) == _lib.MOE_ERR_NULL
    assert b(0, 64, None, None, None, None, None, None, None, None, None) == _lib.MOE_OK


def test_wgrad_ckpt_refusals(lib):
    def w(codes=FAKE, scales=FAKE, a_rows=64, slot=FAKE, div=2, D=FAKE, off=FAKE, E=4, M=128, P=64, Q=64, out=FAKE,
          ws=None):
        return lib.moe_grouped_gemm_wgrad_ckpt(codes, scales, a_rows, slot, div, D, off, E, M, P, Q, out, ws, 0, None)

    assert w(P=48) == _lib.MOE_ERR_UNSUPPORTED
    assert w(Q=60) == _lib.MOE_ERR_UNSUPPORTED
    assert w(Q=1 << 25) == _lib.MOE_ERR_UNSUPPORTED
    assert w(E=256, P=1 << 25, Q=1 << 14, a_rows=1) == _lib.MOE_ERR_UNSUPPORTED
    assert w(E=0) == _lib.MOE_ERR_SHAPE
    assert w(E=257) == _lib.MOE_ERR_UNSUPPORTED
    assert w(div=0) == _lib.MOE_ERR_SHAPE
    assert w(slot=None) == _lib.MOE_ERR_SHAPE  # 64 checkpoint rows, 128 rows
    assert w(a_rows=0) == _lib.MOE_ERR_SHAPE
    assert w(a_rows=-1) == _lib.MOE_ERR_SHAPE
    assert w(a_rows=1 << 25) == _lib.MOE_ERR_UNSUPPORTED
    assert w(off=None) == _lib.MOE_ERR_NULL
    assert w(codes=None) == _lib.MOE_ERR_NULL
    assert w(out=ODD) == _lib.MOE_ERR_ALIGN
    assert w(ws=ODD) == _lib.MOE_ERR_ALIGN
    size = lib.moe_wgrad_ckpt_workspace_bytes
    assert size(4, 2047, 64, 64) == 0 and size(4, 1 << 16, 64, 64) > 0
    assert size(4, 1 << 16, 48, 64) == 0 and size(0, 1 << 16, 64, 64) == 0


def test_routed_layer_refusals(lib):
    S = C.byref(_lib.shape(64, 128, 256, 8, 2))
    full, int8 = _lib.MoeSaved(*([0x1000] * 10)), _lib.MoeSaved8(*([0x1000] * 8))
    big = 1 << 40

    def fwd(shape=S, x=FAKE, idx=FAKE, w=FAKE, wi=FAKE, y=FAKE, saved=None, saved8=None, ws=FAKE, n=big):
        return lib.moe_ffn_fwd_routed(shape, x, idx, w, wi, FAKE, y, saved, saved8, ws, n, None)

    assert fwd(saved=C.byref(full), saved8=C.byref(int8)) == _lib.MOE_ERR_SHAPE
    assert fwd(idx=None) == _lib.MOE_ERR_NULL
    assert fwd(w=ODD) == _lib.MOE_ERR_ALIGN
    assert fwd(wi=None) == _lib.MOE_ERR_NULL
    assert fwd(n=64) == _lib.MOE_ERR_WORKSPACE
    assert fwd(shape=C.byref(_lib.shape(64, 96, 256, 8, 2))) == _lib.MOE_ERR_UNSUPPORTED
    for i in range(8):
        part = _lib.MoeSaved8(*[0 if j == i else 0x1000 for j in range(8)])
        assert fwd(saved8=C.byref(part)) == _lib.MOE_ERR_NULL

    def bwd(shape=S, dy=FAKE, w=FAKE, saved8=int8, dx=FAKE, n=big):
        return lib.moe_ffn_bwd_ckpt(shape, dy, w, None if saved8 is None else C.byref(saved8), FAKE, FAKE, dx, FAKE,
                                    FAKE, FAKE, FAKE, n, None)

    assert bwd(saved8=None) == _lib.MOE_ERR_NULL
    assert bwd(dy=None) == _lib.MOE_ERR_NULL
    assert bwd(w=None) == _lib.MOE_ERR_NULL
    assert bwd(dx=ODD) == _lib.MOE_ERR_ALIGN
    assert bwd(n=64) == _lib.MOE_ERR_WORKSPACE
    for i in range(1, 8):  # group_sizes alone is not read by the backward
        part = _lib.MoeSaved8(*[0 if j == i else 0x1000 for j in range(8)])
        assert bwd(saved8=part) == _lib.MOE_ERR_NULL
    assert lib.moe_workspace_bytes_routed(S, 1) >= 128 * (4 * 256 * 2 + 128 * 2)
    assert lib.moe_workspace_bytes_routed(C.byref(_lib.shape(64, 96, 256, 8, 2)), 0) == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="HIP device"):
        moe.route_scored(2, l)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        moe.route_scored(2, l.half())
    with pytest.raises(ValueError, match="HIP device"):
        moe.ckpt_quantize(l)
    with pytest.raises(TypeError):
        moe.ckpt_dequantize(l, l)
    with pytest.raises(TypeError):
        moe.swiglu_bwd_ckpt(l, l, l)
    with pytest.raises(TypeError):
        moe.grouped_gemm_wgrad_ckpt(l, l, l, l, 2)
