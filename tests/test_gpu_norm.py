"""The norms around the layer, forward and backward, against plain 64-bit formulas and against differences.

Bounds: a row's mean square is a sum of emb positive terms in fp32 (at most 40 additions deep), so a norm's factor is
off by less than 64 * 2^-24; a gradient by 96 * 2^-24 of its terms' magnitudes; a column sum over T rows by
(T + 96) * 2^-24 of its terms' magnitudes; then half a step of the output's type (2^-8 in bf16, 2^-24 in fp32).
"""
import numpy as np
import pytest
import torch

import few_util as fu
import mixture_experts_ffn_group_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32

# rows of one chunk, of 16 lanes, of a wave's, of 128, 256 and 512 lanes, full and not; row counts that leave groups
# empty
SHAPES = [(1, 8), (5, 64), (3, 520), (130, 1088), (7, 2048), (6, 2056), (9, 4096), (1027, 192), (4, 7168), (3, 8192),
          (2, 8200), (3, 16384)]


def _half(t):
    return fu.H if t == BF else fu.U


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(T, emb, dtype, seed):
    g = _gen(seed)
    v = torch.randn((T, emb), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    if T > 2:
        v[1] = 0  # a row of zeros: 0, and a gradient of size eps^-1/2
    return v.to(dtype)


def _weight(emb, kind, seed):
    return None if kind is None else (0.5 + torch.rand(emb, generator=_gen(seed))).to(kind)


def _dev(t):
    return None if t is None else t.to(DEV)


def _check(got, ref, mag, n, dtype):
    """|got - ref| within n * 2^-24 of the terms' magnitudes and half a step of the output's type."""
    assert got.dtype == dtype
    e = np.abs(fu.f64(got) - ref)
    err = n * fu.U * mag
    bound = err + _half(dtype) * (np.abs(ref) + err) + 2.0 ** -133
    assert (e <= bound).all(), f"worst {np.nanmax(e / bound):.2f} of the bound"


@pytest.mark.parametrize("T,emb", SHAPES)
@pytest.mark.parametrize("xt,wt,offset", [(BF, F32, 0.0), (F32, BF, 1.0), (F32, None, 0.0)])
def test_norm_and_its_gradient(T, emb, xt, wt, offset):
    x, w = _rows(T, emb, xt, 1), _weight(emb, wt, 2)
    ref, _ = fu.rms(fu.f64(x), fu.f64(w), offset, EPS)
    y = moe.norm(_dev(x), _dev(w), offset=offset, eps=EPS)
    _check(y, ref, np.abs(ref), 64, BF)
    dy, dres = torch.randn((T, emb), generator=_gen(3)).to(BF), torch.randn((T, emb), generator=_gen(4)).to(xt)
    for r in (dres, None):
        dx, dw = moe.norm_bwd(_dev(dy), _dev(x), _dev(w), offset=offset, eps=EPS, dres=_dev(r))
        gx, gw, mx, mw = fu.norm_grad(fu.f64(dy), fu.f64(x), fu.f64(w), offset, EPS)
        add = 0 if r is None else fu.f64(r)
        _check(dx, add + gx, np.abs(add) + mx, 96, xt)
        assert (dw is None) == (w is None)
        if dw is not None:
            _check(dw, gw, mw, T + 96, F32)


GATES = [(None, F32), ("channel", F32), ("channel", BF), ("token", BF), ("full", F32), ("full", BF)]


def _gate(kind, T, emb, dtype):
    if kind is None:
        return None
    shape = {"channel": (emb,), "token": (T, 1), "full": (T, emb)}[kind]
    v = torch.randn(shape, generator=_gen(5)).to(dtype)
    v.view(-1)[0] = 0  # a closed gate: its gradient is not 0
    return v


def _block_ref(res, y, gate, pw, nw, post, nxt, offset, scale, res_scale):
    z = fu.rms(y, pw, offset, EPS)[0] if post else y
    add = scale * z * (1 if gate is None else gate)
    out = res_scale * res + add
    return z, out, np.abs(res_scale * res) + np.abs(add), fu.rms(out, nw, offset, EPS) if nxt else None


@pytest.mark.parametrize("T,emb", SHAPES)
@pytest.mark.parametrize("gate,gt", GATES)
@pytest.mark.parametrize("post,nxt,xt,wt", [(True, True, BF, F32), (True, False, F32, BF), (False, True, F32, None),
                                            (False, False, BF, None)])
def test_block_out_and_its_gradient(T, emb, gate, gt, post, nxt, xt, wt):
    res, y, gv = _rows(T, emb, xt, 6), _rows(T, emb, BF, 7), _gate(gate, T, emb, gt)
    pw, nw = _weight(emb, wt if post else None, 8), _weight(emb, wt if nxt else None, 9)
    how = dict(post_norm=post, post_weight=_dev(pw), gate=_dev(gv), scale=0.75, res_scale=1.25, next_norm=nxt,
               next_weight=_dev(nw), offset=0.5, eps=EPS)
    r = moe.block_out(_dev(res), _dev(y), **how)
    g64, p64, n64 = fu.f64(gv), fu.f64(pw), fu.f64(nw)
    z, out, mag, xn = _block_ref(fu.f64(res), fu.f64(y), g64, p64, n64, post, nxt, 0.5, 0.75, 1.25)
    _check(r["out"], out, mag, 72, xt)
    if nxt:
        f = np.abs(xn[0] / np.where(out == 0, 1, out))
        _check(r["xn"], xn[0], f * (np.abs(out) + mag) + np.abs(xn[0]) *
               (mag * np.abs(out)).mean(1, keepdims=True) * xn[1] ** 2, 72, BF)
    else:
        assert r["xn"] is None

    dout, dxn = torch.randn((T, emb), generator=_gen(10)).to(xt), torch.randn((T, emb), generator=_gen(11)).to(BF)
    stored = r["out"]
    got = moe.block_out_bwd(_dev(dout), _dev(y), out=stored if nxt else None, dxn=_dev(dxn) if nxt else None, **how)
    d, md = fu.f64(dout), np.abs(fu.f64(dout))
    if nxt:
        gx, gw, mx, mw = fu.norm_grad(fu.f64(dxn), fu.f64(stored), n64, 0.5, EPS)
        d, md = d + gx, md + mx
        if nw is not None:
            _check(got["dnext_weight"], gw, mw, T + 96, F32)
    _check(got["dres"], 1.25 * d, 1.25 * md, 96, xt)
    gg = 1 if g64 is None else g64
    dz, mz, y64 = 0.75 * gg * d, 0.75 * np.abs(gg) * md, fu.f64(y)
    if post:
        dy, dpw, _, _ = fu.norm_grad(dz, y64, p64, 0.5, EPS)
        # what d's own error may add goes through the same terms: md in the place of |d|
        _, _, my, mpw = fu.norm_grad(mz, np.abs(y64), None if p64 is None else np.abs(p64), 0.5, EPS)
        _check(got["dy"], dy, my, 256, BF)
        if pw is not None:
            _check(got["dpost_weight"], dpw, mpw, T + 256, F32)
    else:
        _check(got["dy"], dz, mz, 128, BF)
    if gate is None:
        assert got["dgate"] is None
        return
    dg, mg = 0.75 * d * z, 0.75 * md * np.abs(z)
    if gate == "channel":
        _check(got["dgate"], dg.sum(0), mg.sum(0), T + 256, F32)
    elif gate == "token":
        _check(got["dgate"], dg.sum(1, keepdims=True), mg.sum(1, keepdims=True), 256, F32)
    else:
        _check(got["dgate"], dg, mg, 256, gt)


@pytest.mark.parametrize("T,emb,k", [(1, 64, 1), (5, 520, 3), (33, 2048, 8), (130, 192, 2), (6, 7168, 8), (3, 8200, 64),
                                     (9, 1088, 13), (401, 128, 3), (300, 256, 11), (259, 8, 64)])
@pytest.mark.parametrize("xt", [BF, F32])
def test_block_out_from_expert_rows(T, emb, k, xt):
    g = _gen(12)
    ys = torch.randn((T * k, emb), generator=g).to(BF)
    rows = torch.randperm(T * k, generator=g).to(torch.int32)
    w = torch.rand((T, k), generator=g)
    if T > 4:
        rows[2], rows[7] = -1, T * k  # rows outside add nothing
    res, nw = _rows(T, emb, xt, 13), _weight(emb, F32, 14)
    r = moe.block_out(_dev(res), ys=_dev(ys), slot_row=_dev(rows), topk_w=_dev(w), next_norm=True, next_weight=_dev(nw),
                      want_y=True, eps=EPS)
    y, my = np.zeros((T, emb)), np.zeros((T, emb))
    for q in range(T * k):
        if 0 <= rows[q] < T * k:
            term = float(w.view(-1)[q]) * fu.f64(ys[rows[q]])
            y[q // k] += term
            my[q // k] += np.abs(term)
    _check(r["y"], y, my, k + 1, BF)
    if emb % 64 == 0:  # combine's widths
        assert torch.equal(r["y"], moe.combine(_dev(ys), _dev(rows), _dev(w), T, k))
    out = fu.f64(res) + y
    _check(r["out"], out, np.abs(fu.f64(res)) + my, k + 4, xt)
    p = moe.block_out(_dev(res), ys=_dev(ys), slot_row=_dev(rows), topk_w=_dev(w), post_norm=True, scale=0.5, eps=EPS)
    z, ry = fu.rms(y, None, 0, EPS)
    _check(p["out"], fu.f64(res) + 0.5 * z, np.abs(fu.f64(res)) + ry * (my + np.abs(y)), 64 + 2 * k, xt)
    assert p["y"] is None and p["xn"] is None


def test_gradients_against_differences():
    """The kernels' gradients predict the change of the 64-bit loss sum(dout * out) + sum(dxn * xn) along random
    directions: central differences of step 2^-12, whose error is of the step's square."""
    T, emb = 4, 72
    res, y, gate = _rows(T, emb, F32, 1), _rows(T, emb, BF, 2), _gate("token", T, emb, F32)
    y[1] = 0.5  # no row of zeros here: its curvature is eps^-1
    pw, nw = _weight(emb, F32, 3), _weight(emb, F32, 4)
    dout, dxn = torch.randn((T, emb), generator=_gen(5)), torch.randn((T, emb), generator=_gen(6)).to(BF)
    how = dict(post_norm=True, scale=0.75, res_scale=1.25, next_norm=True, offset=0.5, eps=EPS)
    fwd = moe.block_out(_dev(res), _dev(y), post_weight=_dev(pw), gate=_dev(gate), next_weight=_dev(nw), **how)
    got = moe.block_out_bwd(_dev(dout), _dev(y), out=fwd["out"], dxn=_dev(dxn), post_weight=_dev(pw), gate=_dev(gate),
                            next_weight=_dev(nw), **how)

    def loss(v):
        _, out, _, xn = _block_ref(v[0], v[1], v[2], v[3], v[4], True, True, 0.5, 0.75, 1.25)
        return (fu.f64(dout) * out).sum() + (fu.f64(dxn) * xn[0]).sum()

    vals = [fu.f64(t) for t in (res, y, gate, pw, nw)]
    grads = [fu.f64(got[n]) for n in ("dres", "dy", "dgate", "dpost_weight", "dnext_weight")]
    rng = np.random.default_rng(0)
    for i, (v, g) in enumerate(zip(vals, grads)):
        u = rng.standard_normal(v.shape)
        h = 2.0 ** -12
        up, down = list(vals), list(vals)
        up[i], down[i] = v + h * u, v - h * u
        diff = (loss(up) - loss(down)) / (2 * h)
        # dy is bf16: 2^-8 of each term
        tol = (2.0 ** -8 if i == 1 else 1e-5) * np.abs(g * u).sum() + 1e-4
        assert abs(diff - (g * u).sum()) <= tol, i


def test_aliases_optional_outputs_and_no_rows():
    T, emb = 37, 704
    res, y, w = _dev(_rows(T, emb, F32, 1)), _dev(_rows(T, emb, BF, 2)), _dev(_weight(emb, F32, 3))
    how = dict(post_norm=True, post_weight=w, next_norm=True, next_weight=w, eps=EPS)
    r = moe.block_out(res, y, **how)
    buf = torch.full((T + 2, emb), 9.0, device=DEV)
    buf[:T] = res
    a = moe.block_out(buf[:T], y, out=buf[:T], **how)
    assert torch.equal(buf[:T], r["out"]) and torch.equal(a["xn"], r["xn"]) and (buf[T:] == 9).all()
    dout, dxn = torch.randn((T, emb), device=DEV), torch.randn((T, emb), device=DEV).to(BF)
    full = moe.block_out_bwd(dout, y, out=r["out"], dxn=dxn, **how)
    for n in ("dres", "dy", "dpost_weight", "dnext_weight"):
        one = moe.block_out_bwd(dout, y, out=r["out"], dxn=dxn, need=(n,), **how)
        assert torch.equal(one[n], full[n]) and all(v is None for m, v in one.items() if m != n)
    # no gradient on the residual stream itself
    none = moe.block_out_bwd(None, y, out=r["out"], dxn=dxn, **how)
    zero = moe.block_out_bwd(torch.zeros_like(dout), y, out=r["out"], dxn=dxn, **how)
    assert all(torch.equal(none[n], zero[n]) for n in ("dres", "dy", "dpost_weight", "dnext_weight"))
    # no rows: sums of nothing
    e = moe.block_out_bwd(dout[:0], y[:0], out=res[:0], dxn=dxn[:0], gate=w, **how)
    assert e["dres"].shape == (0, emb) and not e["dgate"].any() and not e["dpost_weight"].any()
    assert not e["dnext_weight"].any()
    dx, dw = moe.norm_bwd(dxn[:0], res[:0], w)
    assert dx.shape == (0, emb) and not dw.any()
    assert moe.norm(res[:0], w).shape == (0, emb) and moe.block_out(res[:0], y[:0])["out"].shape == (0, emb)


def test_infinities_stay_in_their_row_and_repeat_calls_are_equal():
    T, emb = 70, 512
    x, w = _rows(T, emb, F32, 1), _weight(emb, F32, 3)
    clean = moe.norm(_dev(x), _dev(w))
    x[9, 3], x[11, 0] = float("inf"), float("nan")
    y = moe.norm(_dev(x), _dev(w))
    keep = [t for t in range(T) if t not in (9, 11)]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[11]).all()
    dy = torch.randn((T, emb), generator=_gen(4)).to(BF).to(DEV)
    x = _dev(_rows(T, emb, F32, 1))
    a, b = moe.norm_bwd(dy, x, _dev(w)), moe.norm_bwd(dy, x, _dev(w))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_of_forward_and_backward_replays():
    T, emb = 300, 1088
    res, y, w = _dev(_rows(T, emb, BF, 1)), _dev(_rows(T, emb, BF, 2)), _dev(_weight(emb, BF, 3))
    gate = _dev(_gate("channel", T, emb, F32))
    how = dict(post_norm=True, post_weight=w, next_norm=True, next_weight=w, gate=gate, eps=EPS)

    def step(res, y):
        r = moe.block_out(res, y, **how)
        g = moe.block_out_bwd(r["out"], y, out=r["out"], dxn=r["xn"], **how)
        return [r["out"], r["xn"], g["dres"], g["dy"], g["dpost_weight"], g["dgate"], g["dnext_weight"],
                *moe.norm_bwd(r["xn"], res, w)]

    step(res, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(res, y)
    for i in range(4):
        res.copy_(_rows(T, emb, BF, 20 + i))
        y.copy_(_rows(T, emb, BF, 30 + i))
        graph.replay()
        torch.cuda.synchronize()
        ref = step(res.clone(), y.clone())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_more_rows_than_one_grid_dimension_holds():
    """2^21 rows lie along a grid's first dimension; the rest, and none past the last, along the second."""
    T, emb = 2 * 2 ** 21 + 77, 8
    x = torch.randn((T, emb), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(BF)
    y = torch.full((T + 3, emb), 5.0, dtype=BF, device=DEV)
    moe.norm(x, out=y[:T])
    v = x.double()
    ref = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    assert bool(((y[:T].double() - ref).abs() <= (2.0 ** -8 + 64 * fu.U) * ref.abs()).all()) and (y[T:] == 5).all()
    r = moe.block_out(x, ys=x, slot_row=torch.arange(T, dtype=torch.int32, device=DEV),
                      topk_w=torch.ones((T, 1), device=DEV))
    assert torch.equal(r["out"], (x.float() + x.float()).to(BF))
