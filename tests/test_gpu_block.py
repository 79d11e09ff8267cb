"""A transformer block's FFN half run whole: norm, the layer, what joins its output to the residual stream; at decode
on the few-token layer and in training with every gradient, against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import few_util as fu
import mixture_experts_ffn_group_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


def _case(T, emb, mlp, E, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(res=r(T, emb).to(DEV), wi=(r(E, emb, 2 * mlp) / emb ** 0.5).bfloat16().to(DEV),
                wo=(r(E, mlp, emb) / mlp ** 0.5).bfloat16().to(DEV), wr=(r(emb, E) * 0.1).to(DEV),
                w0=(1 + 0.1 * r(emb)).to(DEV), w1=(1 + 0.1 * r(emb)).to(DEV), w2=(1 + 0.1 * r(emb)).to(DEV),
                gate=(0.5 + 0.1 * r(emb)).to(DEV), dout=r(T, emb).to(DEV), dxn=r(T, emb).bfloat16().to(DEV))


@pytest.mark.parametrize("T", [1, 6, 64])
@pytest.mark.parametrize("mx", [False, True])
def test_decode_block(T, mx):
    emb, mlp, E, k = 512, 192, 20, 4
    d = _case(T, emb, mlp, E, T)
    how = dict(post_norm=True, post_weight=d["w1"], gate=d["gate"], next_norm=True, next_weight=d["w2"], eps=EPS)
    xn = moe.norm(d["res"], d["w0"], eps=EPS)
    if mx:
        wq = moe.mx_quantize_expert_weights(d["wi"], d["wo"])
        y, idx, w = moe.ffn_fwd_few_mx(xn, wq, k, wr=d["wr"])
    else:
        y, idx, w = moe.ffn_fwd_few(xn, d["wi"], d["wo"], k, wr=d["wr"])
    r = moe.block_out(d["res"], y, **how)
    ri, rw = fu.route(fu.f64(xn), fu.f64(d["wr"]), None, k)
    assert np.array_equal(idx.cpu().numpy(), ri)
    out = fu.f64(d["res"]) + fu.f64(d["gate"]) * fu.rms(fu.f64(y), fu.f64(d["w1"]), 0, EPS)[0]
    nxt = fu.rms(out, fu.f64(d["w2"]), 0, EPS)[0]
    # fp32 sums of the norm and one addition; half a step of bf16
    assert np.allclose(fu.f64(r["out"]), out, rtol=0, atol=128 * fu.U * np.abs(out).max())
    assert np.linalg.norm(fu.f64(r["xn"]) - nxt) <= fu.H * np.linalg.norm(nxt)
    if not mx:
        yr, err = fu.few(fu.f64(xn), fu.f64(d["wi"]), fu.f64(d["wo"]), ri, fu.f64(w))
        assert (np.abs(fu.f64(y) - yr) <= err).all()


def test_training_block_gradients():
    """The 64-bit block by automatic differentiation on the CPU, routing held fixed; the bf16 roundings between the
    calls (xn, y, dy and the layer's own a, o, dh) leave a relative Frobenius error below 2e-2: about ten roundings of
    2^-9 root mean square each add to under 1 %, and the suite's bound for the layer alone is 1e-2."""
    T, emb, mlp, E, k = 96, 256, 128, 8, 2
    d = _case(T, emb, mlp, E, 3)
    how = dict(post_norm=True, post_weight=d["w1"], gate=d["gate"], scale=0.5, next_norm=True, next_weight=d["w2"],
               eps=EPS)
    xn = moe.norm(d["res"], d["w0"], eps=EPS)
    y, saved = moe.ffn_fwd(xn, d["wi"], d["wo"], k, wr=d["wr"], save=True)
    # the rows combined on the way give the same sum as the layer's y, unrounded
    rows = moe.block_out(d["res"], ys=saved["o"], slot_row=saved["slot_row"], topk_w=saved["topk_w"], want_y=True, **how)
    assert torch.equal(rows["y"], y)
    fwd = moe.block_out(d["res"], y, **how)
    assert float((rows["out"] - fwd["out"]).abs().max()) <= 2.0 ** -7 * float(fwd["out"].abs().max())
    g = moe.block_out_bwd(d["dout"], y, out=fwd["out"], dxn=d["dxn"], **how)
    gl = moe.ffn_bwd(g["dy"], saved, d["wi"], d["wo"], k)
    gr = moe.route_bwd(xn, d["wr"], saved["topk_idx"], saved["topk_w"], gl["dtopk_w"], saved["sorted_slot"],
                       saved["group_offsets"], dx=gl["dx"], want_dbias=False)
    dres, dw0 = moe.norm_bwd(gl["dx"], d["res"], d["w0"], eps=EPS, dres=g["dres"])

    c = {n: d[n].cpu().double().requires_grad_(True) for n in ("res", "wi", "wo", "wr", "w0", "w1", "w2", "gate")}
    rms = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w  # noqa: E731
    x = rms(c["res"], c["w0"])
    idx = saved["topk_idx"].cpu().long()
    w = torch.softmax((x @ c["wr"]).gather(1, idx), dim=1)
    out = torch.zeros((T, emb), dtype=torch.float64)
    for j in range(k):
        h = torch.bmm(x[:, None, :], c["wi"][idx[:, j]])[:, 0]
        a = torch.nn.functional.silu(h[:, :mlp]) * h[:, mlp:]
        out = out + w[:, j:j + 1] * torch.bmm(a[:, None, :], c["wo"][idx[:, j]])[:, 0]
    o = c["res"] + 0.5 * c["gate"] * rms(out, c["w1"])
    loss = (o * d["dout"].cpu().double()).sum() + (rms(o, c["w2"]) * d["dxn"].cpu().double()).sum()
    loss.backward()
    for n, got in (("res", dres), ("wi", gl["dwi"]), ("wo", gl["dwo"]), ("wr", gr["dwr"]), ("w0", dw0),
                   ("w1", g["dpost_weight"]), ("w2", g["dnext_weight"]), ("gate", g["dgate"])):
        ref = c[n].grad
        rel = float((got.cpu().double() - ref).norm() / ref.norm())
        assert rel < 2e-2, (n, rel)
