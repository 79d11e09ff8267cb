"""The norms' gradients where a workgroup takes several sets of rows, as it does in training: 256 workgroups of 512 lanes, a
row in 16 lanes or in whole waves. Each shape has a third, ragged set, so that rows loaded ahead, sums carried on and the
buffers between waves are all used again. The forward's kernels for more than 256 rows are checked on the way."""
import ctypes as C

import numpy as np
import pytest
import torch

import few_util as fu
import mixture_experts_ffn_group_amd as moe
import test_gpu_norm as tn
from mixture_experts_ffn_group_amd import _lib
from test_gpu_norm import BF, DEV, EPS, F32, _dev, _gate, _gen, _rows, _weight

pytestmark = pytest.mark.gpu

# rows, emb, rows of a set: 16 lanes a row; two waves; three waves; five; five of four chunks a lane, nothing loaded ahead
SHAPES = [(2 * 8192 + 45, 192, 32), (2 * 1024 + 9, 1088, 4), (2 * 512 + 3, 2056, 2), (700, 4104, 1), (515, 8200, 1)]
# gate, its type, post norm, next norm, residual's type, weights' type; fp32 with a post norm and a channel gate loads
# nothing ahead
BLOCKS = [(None, F32, True, True, BF, F32), ("channel", F32, True, True, BF, F32), ("channel", BF, True, True, F32, F32),
          ("channel", F32, True, False, F32, BF), ("channel", BF, False, True, F32, None), ("token", BF, True, True, BF, F32),
          ("token", BF, False, False, BF, None), ("full", F32, True, False, F32, BF), ("full", BF, False, True, F32, None)]


@pytest.mark.parametrize("T,emb,per", SHAPES)
@pytest.mark.parametrize("xt,wt,offset", [(BF, F32, 0.0), (F32, BF, 1.0)])
def test_norm_of_many_sets(T, emb, per, xt, wt, offset):
    tn.test_norm_and_its_gradient(T, emb, xt, wt, offset)


@pytest.mark.parametrize("T,emb,per", SHAPES)
@pytest.mark.parametrize("gate,gt,post,nxt,xt,wt", BLOCKS)
def test_block_of_many_sets(T, emb, per, gate, gt, post, nxt, xt, wt):
    tn.test_block_out_and_its_gradient(T, emb, gate, gt, post, nxt, xt, wt)


@pytest.mark.parametrize("T,emb,per", SHAPES)
@pytest.mark.parametrize("gate,xt", [("channel", BF), ("channel", F32), ("token", BF)])
def test_sums_take_every_set_once(T, emb, per, gate, xt):
    """Gradients of 0 but in n <= 96 rows of the second or of the last set: few enough that a row lost or taken twice stands
    out of the bound on the rounding of their sum, (n + 256) 2^-24 of its terms against 1 / n."""
    from_row = 256 * per
    res, y, gv = _rows(T, emb, xt, 6), _rows(T, emb, BF, 7), _gate(gate, T, emb, F32)
    pw, nw = _weight(emb, F32, 8), _weight(emb, F32, 9)
    how = dict(post_norm=True, post_weight=_dev(pw), gate=_dev(gv), next_norm=True, next_weight=_dev(nw), eps=EPS)
    out = moe.block_out(_dev(res), _dev(y), **how)["out"]
    dout, dxn = torch.randn((T, emb), generator=_gen(10)).to(xt), torch.randn((T, emb), generator=_gen(11)).to(BF)
    for t0, t1 in ((from_row, from_row + 3 * per), (T - 5, T)):
        o, n = torch.zeros_like(dout), torch.zeros_like(dxn)
        o[t0:t1], n[t0:t1] = dout[t0:t1], dxn[t0:t1]
        got = moe.block_out_bwd(_dev(o), _dev(y), out=out, dxn=_dev(n), **how)
        zero = np.r_[0:t0, t1:T]
        assert not got["dres"][zero].any() and not got["dy"][zero].any()
        gx, gw, mx, mw = fu.norm_grad(fu.f64(n[t0:t1]), fu.f64(out[t0:t1]), fu.f64(nw), 0, EPS)
        tn._check(got["dnext_weight"], gw, mw, t1 - t0 + 256, F32)
        d, md, g = fu.f64(o[t0:t1]) + gx, np.abs(fu.f64(o[t0:t1])) + mx, fu.f64(gv)[t0:t1] if gate == "token" else fu.f64(gv)
        _, dpw, _, _ = fu.norm_grad(g * d, fu.f64(y[t0:t1]), fu.f64(pw), 0, EPS)
        _, _, _, mpw = fu.norm_grad(np.abs(g) * md, np.abs(fu.f64(y[t0:t1])), fu.f64(pw), 0, EPS)
        tn._check(got["dpost_weight"], dpw, mpw, t1 - t0 + 256, F32)
        if gate == "channel":
            z = fu.rms(fu.f64(y[t0:t1]), fu.f64(pw), 0, EPS)[0]
            tn._check(got["dgate"], (d * z).sum(0), (md * np.abs(z)).sum(0), t1 - t0 + 256, F32)


@pytest.mark.parametrize("T,emb,per", [(5, 64, 32), *SHAPES])
@pytest.mark.parametrize("xt", [BF, F32])
def test_gradients_in_place(T, emb, per, xt):
    """dx may be dres itself, dres dout itself: the same bits as out of place, whatever has been loaded ahead."""
    x, y, w = _dev(_rows(T, emb, xt, 1)), _dev(_rows(T, emb, BF, 2)), _dev(_weight(emb, F32, 3))
    d = torch.randn((T, emb), generator=_gen(4)).to(xt).to(DEV)
    dxn = torch.randn((T, emb), generator=_gen(5)).to(BF).to(DEV)
    ty = _lib.MOE_F32 if xt == F32 else _lib.MOE_BF16
    lib, p = _lib.lib(), lambda t: C.c_void_p(t.data_ptr())
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)

    ref, ref_w = moe.norm_bwd(dxn, x, w, dres=d, eps=EPS)
    ws = torch.empty(lib.moe_block_out_bwd_workspace_bytes(T, emb), dtype=torch.uint8, device=DEV)
    buf, dw = torch.cat([d, d[:2]]), torch.empty(emb, device=DEV)
    assert lib.moe_norm_bwd(T, emb, p(dxn), p(x), ty, p(w), _lib.MOE_F32, 0.0, EPS, p(buf), p(buf), p(dw), p(ws), ws.numel(),
                            stream) == _lib.MOE_OK
    assert torch.equal(buf[:T], ref) and torch.equal(dw, ref_w) and torch.equal(buf[T:], d[:2])

    how = dict(post_norm=True, post_weight=w, gate=w, next_norm=True, next_weight=w, eps=EPS)
    out = moe.block_out(x, y, **how)["out"]
    ref = moe.block_out_bwd(d, y, out=out, dxn=dxn, **how)
    b = _lib.MoeBlock(x_type=ty, weight_type=_lib.MOE_F32, gate_mode=_lib.MOE_GATE_CHANNEL, gate_type=_lib.MOE_F32, post=1,
                      offset=0.0, eps=EPS, scale=1.0, res_scale=1.0, post_weight=w.data_ptr(), next_weight=w.data_ptr(),
                      gate=w.data_ptr())
    buf, dy = torch.cat([d, d[:2]]), torch.empty_like(y)
    sums = [torch.empty(emb, device=DEV) for _ in range(3)]
    assert lib.moe_block_out_bwd(T, emb, C.byref(b), p(buf), p(y), p(out), p(dxn), p(buf), p(dy), p(sums[0]), p(sums[1]),
                                 p(sums[2]), p(ws), ws.numel(), stream) == _lib.MOE_OK
    assert torch.equal(buf[:T], ref["dres"]) and torch.equal(dy, ref["dy"]) and torch.equal(buf[T:], d[:2])
    for got, n in zip(sums, ("dpost_weight", "dnext_weight", "dgate")):
        assert torch.equal(got, ref[n])
