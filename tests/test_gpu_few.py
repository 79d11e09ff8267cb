"""The layer for a few tokens against a plain 64-bit implementation: router, bf16 and MXFP8 weights, given routings,
masks, empty and repeated experts, graphs, streams. Tolerances are the bounds few_util derives."""
import numpy as np
import pytest
import torch

import few_util as fu
import mixture_experts_ffn_group_amd as moe
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# T, emb, mlp, E, k: one token, one expert, k = E, more than one tile of 16 rows an expert, odd 64-column tails,
# experts past one wave, many slices
SHAPES = [(1, 64, 64, 1, 1), (1, 2048, 768, 128, 8), (5, 1088, 448, 60, 4), (16, 128, 64, 4, 4), (17, 192, 128, 1, 1),
          (64, 64, 320, 3, 3), (33, 192, 128, 256, 8), (64, 128, 256, 8, 2), (3, 320, 2048, 70, 64), (64, 576, 192, 160, 8),
          # few slices and a long contraction: the products in kernels of their own, cut
          (50, 1088, 64, 3, 2), (64, 2112, 128, 1, 1), (7, 5248, 64, 16, 3), (4, 1536, 192, 5, 2),
          # tiles of 32 rows, half-filled ones too, in slices of 128 and of 64 columns
          (40, 192, 2368, 8, 8), (49, 1024, 320, 3, 1), (64, 320, 192, 4, 1), (64, 64, 128, 70, 64),
          # 192 workgroups at emb 4096 (bf16: cut), 390 of 128
          (3, 4096, 1024, 16, 4), (40, 64, 704, 65, 2)]


def _bf(t):
    return t.to(torch.bfloat16)


def _inputs(T, emb, mlp, E, k, seed=0, bias=False):
    g = torch.Generator().manual_seed(seed + 7 * T + emb)
    d = dict(x=_bf(torch.randn((T, emb), generator=g)), wi=_bf(torch.randn((E, emb, 2 * mlp), generator=g) / emb ** 0.5),
             wo=_bf(torch.randn((E, mlp, emb), generator=g) / mlp ** 0.5), wr=torch.randn((emb, E), generator=g) * 0.05,
             bias=torch.randn(E, generator=g) * 0.1 if bias else None)
    return d, {n: None if v is None else v.to(DEV) for n, v in d.items()}


def _mx_values(wq, name):
    """64-bit values [E, K, N] of MXFP8 codes and scales."""
    codes, scales = wq[name + "_codes"].cpu().numpy(), wq[name + "_scales"].cpu().numpy()
    table = np.array([oracle.e4m3_value(c) for c in range(256)])
    E, N, K = codes.shape
    s = np.exp2(scales[..., :2].astype(np.float64) - 127).transpose(0, 2, 1, 3).reshape(E, N, K // 32)
    return (table[codes] * np.repeat(s, 32, axis=2)).transpose(0, 2, 1)


def _close(got, ref, err):
    got = fu.f64(got)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > err
    assert not bad.any(), f"{bad.sum()} elements past the bound, worst {np.max(np.abs(got - ref) / err):.2f} of it"
    # all elements at half a step at once would give 2^-8
    assert np.linalg.norm(got - ref) <= 2.0 ** -8 * np.linalg.norm(ref) + 1e-30


@pytest.mark.parametrize("T,emb,mlp,E,k", SHAPES)
@pytest.mark.parametrize("bias", [False, True])
def test_layer_with_its_router(T, emb, mlp, E, k, bias):
    h, d = _inputs(T, emb, mlp, E, k, bias=bias)
    y, idx, w = moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], k, wr=d["wr"], bias=d["bias"])
    ri, rw = fu.route(fu.f64(h["x"]), fu.f64(h["wr"]), fu.f64(h["bias"]), k)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.allclose(fu.f64(w), rw, rtol=4 * fu.U, atol=0)
    _close(y, *fu.few(fu.f64(h["x"]), fu.f64(h["wi"]), fu.f64(h["wo"]), ri, fu.f64(w)))


@pytest.mark.parametrize("T,emb,mlp,E,k", SHAPES)
def test_given_routing_gives_the_same_bits_and_mx_weights_their_values(T, emb, mlp, E, k):
    h, d = _inputs(T, emb, mlp, E, k, seed=1)
    y, idx, w = moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], k, wr=d["wr"])
    ri = torch.full((T, k), -1, dtype=torch.int32, device=DEV).copy_(idx)
    y2, i2, w2 = moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], topk_idx=ri, topk_w=w)
    assert torch.equal(y, y2) and i2 is ri and w2 is w
    wq = moe.mx_quantize_expert_weights(d["wi"], d["wo"])
    ym, im, wm = moe.ffn_fwd_few_mx(d["x"], wq, k, wr=d["wr"])
    assert torch.equal(im, idx) and torch.equal(wm, w)
    _close(ym, *fu.few(fu.f64(h["x"]), _mx_values(wq, "wi"), _mx_values(wq, "wo"), idx.cpu().numpy(), fu.f64(w)))
    ym2 = moe.ffn_fwd_few_mx(d["x"], wq, topk_idx=idx, topk_w=w)[0]
    assert torch.equal(ym, ym2)


def test_agrees_with_the_layer_for_many_tokens():
    """Same routing, same weights: both are within the bounds of the same 64-bit layer (bf16 roundings of a and o in
    the other: its own tests' 1e-2)."""
    h, d = _inputs(40, 512, 384, 32, 4, seed=2)
    idx, w = moe.route(4, d["x"], d["wr"])
    few = moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], topk_idx=idx, topk_w=w)[0]
    many = moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w)[0]
    assert float((few.double() - many.double()).norm() / many.double().norm()) < 1e-2


def test_skewed_load_every_token_on_the_same_experts():
    T, emb, mlp, E, k = 61, 192, 192, 12, 3
    h, d = _inputs(T, emb, mlp, E, k, seed=3)
    idx = torch.tensor([[7, 0, 11]] * T, dtype=torch.int32)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(1))
    y = moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], topk_idx=idx.to(DEV), topk_w=w.to(DEV))[0]
    _close(y, *fu.few(fu.f64(h["x"]), fu.f64(h["wi"]), fu.f64(h["wo"]), idx.numpy(), fu.f64(w)))


def test_picks_out_of_range_take_no_part_and_repeated_ones_count_twice():
    T, emb, mlp, E, k = 9, 128, 128, 5, 4
    h, d = _inputs(T, emb, mlp, E, k, seed=4)
    idx = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    idx[0] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31])
    idx[1] = 3
    idx[2, 1] = 255
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(3)) + 0.1
    w[2, 1] = float("nan")  # a weight without a part
    ws = torch.full((moe.workspace_bytes_few(T, emb, mlp, E, k),), 0xff, dtype=torch.uint8, device=DEV)  # NaN
    y = moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], topk_idx=idx.to(DEV), topk_w=w.to(DEV), workspace=ws)[0]
    wn = np.nan_to_num(fu.f64(w))
    ref, err = fu.few(fu.f64(h["x"]), fu.f64(h["wi"]), fu.f64(h["wo"]), idx.numpy(), wn)
    assert (ref[0] == 0).all() and torch.equal(y[0], torch.zeros_like(y[0]))
    _close(y, ref, err)


def test_masked_experts_ties_and_rows_of_nan():
    T, emb, mlp, E, k = 12, 256, 64, 130, 6
    h, d = _inputs(T, emb, mlp, E, k, seed=5)
    wr = h["wr"].clone()
    wr[:, 100] = wr[:, 3]          # equal logits: the lower id first
    wr[:, 64:70] = wr[:, :1]
    bias = torch.zeros(E)
    bias[10:40] = -float("inf")
    bias[40] = float("nan")
    bias[100] = bias[3] = 20
    h["x"][4] = 0                  # all logits equal but for the bias
    h["x"][7, 9] = float("nan")    # every logit NaN: the k lowest ids, weights and y NaN
    ri, rw = fu.route(fu.f64(h["x"]), fu.f64(wr), fu.f64(bias), k)
    y, idx, w = moe.ffn_fwd_few(h["x"].to(DEV), d["wi"], d["wo"], k, wr=wr.to(DEV), bias=bias.to(DEV))
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.allclose(fu.f64(w), rw, rtol=4 * fu.U, atol=0, equal_nan=True) and np.isnan(rw[7]).all()
    assert torch.isnan(y[7]).all()
    keep = [t for t in range(T) if t != 7]
    ref, err = fu.few(fu.f64(h["x"])[keep], fu.f64(h["wi"]), fu.f64(h["wo"]), ri[keep], fu.f64(w)[keep])
    _close(y[keep], ref, err)
    # all experts masked: weights 0, y 0, picks distinct and in range
    y, idx, w = moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], k, wr=wr.to(DEV),
                                bias=torch.full((E,), -float("inf"), device=DEV))
    assert np.array_equal(idx.cpu().numpy(), np.tile(np.arange(k), (T, 1))) and not w.any() and not y.any()


@pytest.mark.parametrize("mx", [False, True])
def test_no_tokens_and_rows_behind_the_last(mx):
    T, emb, mlp, E, k = 6, 192, 64, 9, 2
    h, d = _inputs(T, emb, mlp, E, k, seed=6)
    wq = moe.mx_quantize_expert_weights(d["wi"], d["wo"])
    f = (lambda x, **kw: moe.ffn_fwd_few_mx(x, wq, **kw)) if mx else \
        (lambda x, **kw: moe.ffn_fwd_few(x, d["wi"], d["wo"], **kw))
    y, idx, w = f(d["x"][:0], k=k, wr=d["wr"])
    assert y.shape == (0, emb) and idx.shape == (0, k)
    ref = f(d["x"], k=k, wr=d["wr"])[0]
    buf = torch.full((T + 3, emb), 7.0, dtype=torch.bfloat16, device=DEV)
    n = moe.workspace_bytes_few(T, emb, mlp, E, k)
    ws = torch.full((n + 64,), 0xff, dtype=torch.uint8, device=DEV)
    f(d["x"], k=k, wr=d["wr"], out=buf[:T], workspace=ws[:n])
    assert torch.equal(buf[:T], ref) and (buf[T:] == 7).all() and (ws[n:] == 0xff).all()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 7, 40])
def test_graph_replays_equal_eager(T, mx):
    emb, mlp, E, k = 320, 192, 24, 4
    h, d = _inputs(T, emb, mlp, E, k, seed=8)
    wq = moe.mx_quantize_expert_weights(d["wi"], d["wo"])

    def f(x, **kw):
        if mx:
            return moe.ffn_fwd_few_mx(x, wq, k, wr=d["wr"], **kw)
        return moe.ffn_fwd_few(x, d["wi"], d["wo"], k, wr=d["wr"], **kw)

    x = d["x"].clone()
    f(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, idx, w = f(x)
    gen = torch.Generator().manual_seed(9)
    for _ in range(4):
        xr = _bf(torch.randn((T, emb), generator=gen)).to(DEV)
        x.copy_(xr)
        g.replay()
        torch.cuda.synchronize()
        ye, ie, we = f(xr)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(idx, ie) and torch.equal(w, we)


def test_two_streams_and_repeated_calls_give_the_same_bits():
    h, d = _inputs(31, 448, 256, 40, 5, seed=10)
    f = lambda: moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], 5, wr=d["wr"])  # noqa: E731
    ref = f()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        with torch.cuda.stream(s[i % 2]):
            outs.append(f())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_disabled_experts_weights_may_hold_anything():
    """With fewer enabled experts than picks, disabled ones are picked with weight 0; what their weights hold (NaN,
    infinities) does not reach y."""
    T, emb, mlp, E, k = 20, 192, 64, 6, 5
    h, d = _inputs(T, emb, mlp, E, k, seed=11)
    bias = torch.tensor([0.0, -float("inf"), 0.0, -float("inf"), 0.0, float("nan")])
    for e, v in ((1, float("nan")), (3, float("inf")), (5, float("nan"))):
        d["wi"][e], d["wo"][e] = v, v
    for n in (T, 3):
        y, idx, w = moe.ffn_fwd_few(d["x"][:n], d["wi"], d["wo"], k, wr=d["wr"], bias=bias.to(DEV))
        ri, rw = fu.route(fu.f64(h["x"])[:n], fu.f64(h["wr"]), fu.f64(bias), k)
        assert np.array_equal(idx.cpu().numpy(), ri) and (ri[:, 3:] == [1, 3]).all() and (rw[:, 3:] == 0).all()
        _close(y, *fu.few(fu.f64(h["x"])[:n], fu.f64(h["wi"]), fu.f64(h["wo"]), ri, fu.f64(w)))


def test_swiglu_past_bf16_is_infinite_not_nan():
    """silu(g) * u past bf16's range: with positive down weights the output is +inf, as from a rounded to bf16."""
    emb = mlp = 64
    x = torch.ones((2, emb), dtype=torch.bfloat16, device=DEV)
    wi = torch.full((1, emb, 2 * mlp), 2.0 ** 58, dtype=torch.bfloat16, device=DEV)  # g = u = 2^64
    wo = torch.ones((1, mlp, emb), dtype=torch.bfloat16, device=DEV)
    idx, w = torch.zeros((2, 1), dtype=torch.int32, device=DEV), torch.ones((2, 1), device=DEV)
    x[1] = 2.0 ** -58  # g = u = 64: finite beside it
    y = moe.ffn_fwd_few(x, wi, wo, topk_idx=idx, topk_w=w)[0]
    assert torch.equal(y[0], torch.full_like(y[0], float("inf")))
    assert torch.equal(y[1], torch.full_like(y[1], 64.0 * 64 * mlp))


def test_experts_of_zero_weights_give_zeros():
    h, d = _inputs(5, 192, 128, 6, 2, seed=9)
    d["wi"][2:4] = 0
    d["wo"][4] = 0
    idx = torch.tensor([[2, 3], [3, 4], [4, 2], [2, 2], [0, 4]], dtype=torch.int32, device=DEV)
    w = torch.ones((5, 2), device=DEV)
    for y in (moe.ffn_fwd_few(d["x"], d["wi"], d["wo"], topk_idx=idx, topk_w=w)[0],
              moe.ffn_fwd_few_mx(d["x"], moe.mx_quantize_expert_weights(d["wi"], d["wo"]), topk_idx=idx, topk_w=w)[0]):
        assert not y[:4].any() and y[4].any() and torch.isfinite(y).all()


@pytest.mark.parametrize("mx", [False, True])
def test_largest_expert_past_32_bit_offsets(mx):
    """emb 16384, mlp 65472, the second of two experts: its weights start past 2^32 bytes (MXFP8: past 2^31)."""
    T, emb, mlp = 3, 16384, 65472
    g = torch.Generator(device=DEV).manual_seed(5)
    wi = torch.empty((2, emb, 2 * mlp), dtype=torch.bfloat16, device=DEV).normal_(0, emb ** -0.5, generator=g)
    wo = torch.empty((2, mlp, emb), dtype=torch.bfloat16, device=DEV).normal_(0, mlp ** -0.5, generator=g)
    x = torch.empty((T, emb), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    idx, w = torch.ones((T, 1), dtype=torch.int32, device=DEV), torch.tensor([[0.5], [1.0], [0.25]], device=DEV)
    if mx:
        wq = moe.mx_quantize_expert_weights(wi, wo)
        y = moe.ffn_fwd_few_mx(x, wq, topk_idx=idx, topk_w=w)[0]
        s = {n: torch.exp2(wq[n + "_scales"][1, ..., :2].double() - 127).transpose(0, 1) for n in ("wi", "wo")}

        def values(n, lo, hi, k0, k1):  # [N rows, K] of the expert: rows lo..hi, K k0..k1
            c = wq[n + "_codes"][1, lo:hi, k0:k1].view(torch.float8_e4m3fn).double()
            sc = s[n][lo:hi, k0 // 64:k1 // 64].reshape(hi - lo, -1)
            return c * torch.repeat_interleave(sc, 32, dim=1)
        cols = lambda lo, hi: values("wi", lo, hi, 0, emb).T
        rows = lambda lo, hi: values("wo", 0, emb, lo, hi).T
    else:
        y = moe.ffn_fwd_few(x, wi, wo, topk_idx=idx, topk_w=w)[0]
        cols = lambda lo, hi: wi[1, :, lo:hi].double()
        rows = lambda lo, hi: wo[1, lo:hi].double()
    ref, err = torch.zeros((T, emb), dtype=torch.float64, device=DEV), torch.zeros((T, emb), dtype=torch.float64, device=DEV)
    xd = x.double()
    for m in range(0, mlp, 3968):  # 16.5 chunks of whole 64s
        n = min(m + 3968, mlp)
        gate, up, down = cols(m, n), cols(mlp + m, mlp + n), rows(m, n)
        gv, uv = xd @ gate, xd @ up
        dg, du = ((emb + 16) * fu.U * (xd.abs() @ v.abs()) for v in (gate, up))
        sv = torch.nn.functional.silu(gv)
        a = sv * uv
        da = 1.1 * dg * uv.abs() + sv.abs() * du + 1.1 * dg * du + a.abs() * (2.0 ** -16 + 2.0 ** -19)
        ref += a @ down
        err += da @ down.abs() + (mlp + 16) * fu.U * ((a.abs() + da) @ down.abs())
        err += (mlp // 64 + 17) * fu.U * (a.abs() @ down.abs())
    ref, err = ref * w.double(), err * w.double()
    _close(y, ref.cpu().numpy(), (err + fu.H * (ref.abs() + err)).cpu().numpy())
