"""Host validation of the few-token layer and of the norms around the layer: everything here is refused (or has
nothing to do) before any HIP call, so it runs without a GPU."""
import ctypes as C

import pytest
import torch

import mixture_experts_ffn_group_amd as moe
from mixture_experts_ffn_group_amd import _lib

OK, NULL, SHAPE, UNSUP, WS, _, ALIGN = range(7)
P, ODD = C.c_void_p(0x1000), C.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def _shape(T=4, emb=128, mlp=256, E=8, k=2):
    return C.byref(_lib.shape(T, emb, mlp, E, k))


FEW = dict(x=P, wr=P, bias=None, idx=P, w=P, wi=P, wo=P, y=P, ws=P, n=1 << 40)


@pytest.mark.parametrize("shape,change,status", [
    (dict(T=65), {}, UNSUP),
    (dict(T=-1), {}, SHAPE),
    (dict(emb=96), {}, UNSUP),
    (dict(mlp=32), {}, UNSUP),
    (dict(E=257), {}, UNSUP),
    (dict(k=9), {}, SHAPE),
    (dict(T=64, emb=64, mlp=1 << 23, E=256, k=64), {}, UNSUP),  # more workgroups than a grid holds
    ({}, dict(x=None), NULL),
    ({}, dict(x=ODD), ALIGN),
    ({}, dict(wr=ODD), ALIGN),
    ({}, dict(bias=ODD), ALIGN),
    ({}, dict(wr=None, bias=P), SHAPE),
    ({}, dict(idx=None), NULL),
    ({}, dict(w=None), NULL),
    ({}, dict(wi=None), NULL),
    ({}, dict(wo=ODD), ALIGN),
    ({}, dict(y=None), NULL),
    ({}, dict(ws=None), NULL),
    ({}, dict(n=16), WS),
    (dict(T=0), dict(x=None, wi=None, wo=None, y=None, ws=None, n=0, idx=None, w=None), OK),
])
def test_few_refusals(lib, shape, change, status):
    a = {**FEW, **change}
    s = _shape(**shape)
    got = lib.moe_ffn_fwd_few(s, a["x"], a["wr"], a["bias"], a["idx"], a["w"], a["wi"], a["wo"], a["y"], a["ws"], a["n"],
                              None)
    assert got == status and (status == OK) == (lib.moe_last_error_detail() == b"")
    got = lib.moe_ffn_fwd_few_mx(s, a["x"], a["wr"], a["bias"], a["idx"], a["w"], a["wi"], P, a["wo"], P, a["y"],
                                 a["ws"], a["n"], None)
    assert got == status


def test_few_mx_needs_its_scales(lib):
    for c, d in ((None, P), (P, None), (ODD, P), (P, ODD)):
        st = lib.moe_ffn_fwd_few_mx(_shape(), P, P, None, P, P, P, c, P, d, P, P, 1 << 40, None)
        assert st == (ALIGN if ODD in (c, d) else NULL)


def test_few_workspace(lib):
    one = lib.moe_workspace_bytes_few(_shape(T=1))
    assert 0 < one <= lib.moe_workspace_bytes_few(_shape(T=64))
    assert lib.moe_workspace_bytes_few(_shape(T=65)) == 0 and lib.moe_workspace_bytes_few(_shape(emb=96)) == 0
    # the shares of S = 512 rows over emb = 7168, and no more than a share per 64 columns of mlp
    big = lib.moe_workspace_bytes_few(_shape(T=64, emb=7168, mlp=2048, E=256, k=8))
    assert 512 * 7168 * 4 <= big <= 512 * 32 * 7168 * 4 + (64 << 20)
    assert moe.workspace_bytes_few(1, 128, 256, 8, 2) == one


def _norm(lib, T=4, emb=64, x=P, xt=0, w=P, wt=0, off=0.0, eps=1e-6, y=P):
    return lib.moe_norm(T, emb, x, xt, w, wt, off, eps, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), UNSUP), (dict(emb=0), SHAPE), (dict(emb=-8), SHAPE), (dict(emb=12), UNSUP),
    (dict(emb=16392), UNSUP), (dict(x=None), NULL), (dict(x=ODD), ALIGN), (dict(xt=2), SHAPE), (dict(w=ODD), ALIGN),
    (dict(wt=5), SHAPE), (dict(off=float("inf")), SHAPE), (dict(off=float("nan")), SHAPE), (dict(eps=0.0), SHAPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(y=None), NULL),
    (dict(y=ODD), ALIGN), (dict(T=0, x=None, y=None), OK), (dict(T=0, w=None, wt=9), OK)])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(dx=None), NULL), (dict(dres=ODD), ALIGN), (dict(dw=ODD), ALIGN),
    (dict(ws=None), NULL), (dict(n=8), WS), (dict(emb=20), UNSUP), (dict(eps=0.0), SHAPE)])
def test_norm_bwd_refusals(lib, kw, status):
    a = dict(T=4, emb=64, dy=P, x=P, w=P, eps=1e-6, dres=P, dx=P, dw=P, ws=P, n=1 << 30, **{})
    a.update(kw)
    assert lib.moe_norm_bwd(a["T"], a["emb"], a["dy"], a["x"], 0, a["w"], 0, 0.0, a["eps"], a["dres"], a["dx"], a["dw"],
                            a["ws"], a["n"], None) == status


def _block(**kw):
    b = dict(x_type=0, weight_type=0, gate_mode=0, gate_type=0, post=1, offset=0.0, eps=1e-6, scale=1.0, res_scale=1.0,
             post_weight=0x1000, next_weight=0x1000, gate=None)
    b.update(kw)
    return C.byref(_lib.MoeBlock(**b))


BAD_BLOCKS = [
    (dict(x_type=3), SHAPE), (dict(weight_type=3), SHAPE), (dict(gate_mode=4), SHAPE), (dict(gate_mode=-1), SHAPE),
    (dict(gate=0x1000), SHAPE), (dict(gate_mode=1), NULL), (dict(gate_mode=2, gate=0x1004), ALIGN),
    (dict(gate_mode=3, gate=0x1000, gate_type=2), SHAPE), (dict(post=0), SHAPE), (dict(eps=0.0), SHAPE),
    (dict(offset=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(res_scale=float("nan")), SHAPE),
    (dict(post_weight=0x1008), ALIGN), (dict(next_weight=0x1008), ALIGN)]


@pytest.mark.parametrize("kw,status", BAD_BLOCKS)
def test_block_structure_refusals(lib, kw, status):
    b = _block(**kw)
    assert lib.moe_block_out(4, 64, b, P, P, 0, None, None, None, P, P, None, None) == status
    assert lib.moe_block_out_bwd(4, 64, b, P, P, P, P, P, P, None, None, None, None, 0, None) == status


def test_block_out_refusals(lib):
    b, f = _block(), lib.moe_block_out
    assert f(4, 64, None, P, P, 0, None, None, None, P, P, None, None) == NULL
    assert f(4, 64, b, None, P, 0, None, None, None, P, P, None, None) == NULL
    assert f(4, 64, b, P, P, 0, None, None, None, None, P, None, None) == NULL
    assert f(4, 64, b, P, P, 0, None, None, None, P, ODD, None, None) == ALIGN
    assert f(4, 60, b, P, P, 0, None, None, None, P, P, None, None) == UNSUP
    for i in range(4):  # y with any of ys, slot_row, topk_w, y_out
        e = [P if i == j else None for j in range(4)]
        assert f(4, 64, b, P, P, 2, e[0], e[1], e[2], P, P, e[3], None) == SHAPE
    assert f(4, 64, b, P, None, 0, P, P, P, P, P, None, None) == SHAPE
    assert f(4, 64, b, P, None, 65, P, P, P, P, P, None, None) == UNSUP
    assert f(1 << 30, 64, b, P, None, 2, P, P, P, P, P, None, None) == UNSUP
    assert f(4, 64, b, P, None, 2, None, P, P, P, P, None, None) == NULL
    assert f(4, 64, b, P, None, 2, P, None, P, P, P, None, None) == NULL
    assert f(4, 64, b, P, None, 2, P, P, ODD, P, P, None, None) == ALIGN
    assert f(0, 64, b, None, None, 0, None, None, None, None, None, None, None) == OK


def test_block_out_bwd_refusals(lib):
    f = lib.moe_block_out_bwd
    n = 1 << 40

    def call(b=None, dout=P, y=P, out=P, dxn=P, dres=P, dy=P, dp=None, dn=None, dg=None, ws=None, size=0):
        return f(4, 64, b or _block(), dout, y, out, dxn, dres, dy, dp, dn, dg, ws, size, None)

    assert call(dxn=None) == SHAPE                       # out without dxn
    assert call(dxn=None, out=None, dn=P, ws=P, size=n) == SHAPE
    assert call(out=None) == NULL
    assert call(dout=None, dxn=None, out=None) == NULL   # no gradient at all
    assert call(y=None) == NULL                          # the norm after the layer reads y
    assert call(b=_block(post=0, post_weight=None), dp=P, ws=P, size=n) == SHAPE
    assert call(dg=P) == SHAPE
    assert call(dp=P) == NULL and call(dp=P, ws=P, size=64) == WS
    assert call(b=_block(gate_mode=1, gate=0x1000), dg=P) == NULL   # a channel gate's gradient needs the workspace
    assert call(dres=ODD) == ALIGN and call(dy=ODD) == ALIGN


def test_binding_refusals():
    """The binding checks what the library cannot see: types, devices, shapes."""
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="HIP device"):
        moe.norm(x)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        moe.norm(x.half())
    with pytest.raises(ValueError, match="HIP device"):
        moe.ffn_fwd_few(x.bfloat16(), None, None, 2)
    with pytest.raises(ValueError, match="2 dimensions"):
        moe.ffn_fwd_few(None, None, None, 2)
    with pytest.raises(ValueError, match="dout, or dxn and out"):
        moe.block_out_bwd(None)
