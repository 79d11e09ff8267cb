"""The layer on a given routing, its 8-bit saved set, and a training step of the whole set of calls: route_scored,
ffn_fwd_routed, ffn_bwd_ckpt, route_scored_bwd.

What has to be equal bit for bit is compared so: the forward with any saved set against ffn_fwd on the same routing,
and the 8-bit h against the fp32 h of the full set, quantized on the host. Gradients from the 8-bit set are compared
with a 64-bit evaluation at the very values the set holds; their roundings (du, dh, do, a and the outputs, half a
bf16 step, 2^-9 of a value at most, each) leave a relative Frobenius error below 1e-2, the suite's bound for bf16
outputs.
"""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_group_amd as moe
import scored_util as su
import workloads
from parity_util import errors

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
REL = 1e-2


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _case(T, emb, mlp, E, k, seed, sigma=0.05):
    wl = workloads.custom(T, emb, mlp, E, k, seed=seed, sigma_w=sigma, backward=True)
    d = workloads.make_inputs(wl)
    return {n: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for n, v in d.items()}


SHAPES = [(1, 64, 64, 1, 1), (3, 64, 64, 8, 3), (200, 128, 192, 8, 2), (515, 192, 320, 37, 5), (700, 256, 128, 4, 4),
          (1000, 320, 576, 12, 3)]


@pytest.mark.parametrize("T,emb,mlp,E,k", SHAPES)
def test_routed_forward_equals_ffn_fwd(T, emb, mlp, E, k):
    d = _case(T, emb, mlp, E, k, T)
    y, full = moe.ffn_fwd(d["x"], d["wi"], d["wo"], k, wr=d["wr"], save=True)
    idx, w = moe.route(k, d["x"], d["wr"])
    for save in (None, "full", "int8"):
        yr, saved = moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, save=save)
        assert _same_bits(yr, y), save
        if save == "full":
            for n in ("group_sizes", "group_offsets", "sorted_slot", "slot_row", "xs", "h", "a", "o"):
                assert _same_bits(saved[n], full[n]), n
            ref = moe.ffn_bwd(d["dy"], full, d["wi"], d["wo"], k)
            got = moe.ffn_bwd(d["dy"], saved, d["wi"], d["wo"], k)
            for n in ref:
                assert _same_bits(got[n], ref[n]), n
        if save == "int8":
            xc, xs = su.ckpt_quantize(d["x"].cpu().double().numpy())
            hc, hs = su.ckpt_quantize(full["h"].cpu().double().numpy())
            for n, ref in (("x_codes", xc), ("x_scales", xs), ("h_codes", hc), ("h_scales", hs)):
                assert np.array_equal(saved[n].cpu().numpy(), ref), n
            assert _same_bits(saved["sorted_slot"], full["sorted_slot"])


def _bwd_ref(d, saved, k):
    """64-bit gradients at the x and h the 8-bit set holds: dx, dwi, dwo, dtopk_w."""
    x = su.ckpt_values(saved["x_codes"].cpu().numpy(), saved["x_scales"].cpu().numpy())
    h = su.ckpt_values(saved["h_codes"].cpu().numpy(), saved["h_scales"].cpu().numpy())
    wi, wo = d["wi"].cpu().double().numpy(), d["wo"].cpu().double().numpy()
    dy = d["dy"].cpu().double().numpy()
    w = saved["topk_w"].cpu().double().numpy().reshape(-1)
    slot, off = saved["sorted_slot"].cpu().numpy(), saved["group_offsets"].cpu().numpy()
    E, emb, n2 = wi.shape
    mlp = n2 // 2
    T = dy.shape[0]
    dx, dwi, dwo, dw = np.zeros((T, emb)), np.zeros_like(wi), np.zeros_like(wo), np.zeros(T * k)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        q = slot[r]
        t = q // k
        g, u = h[r, :mlp], h[r, mlp:]
        s = 1 / (1 + np.exp(-g))
        a = g * s * u
        du = dy[t] @ wo[e].T
        dw[q] = (a * du).sum(axis=1)
        da = du * w[q][:, None]
        dh = np.concatenate([da * u * s * (1 + g * (1 - s)), da * g * s], axis=1)
        dwi[e] = x[t].T @ dh
        dwo[e] = a.T @ (dy[t] * w[q][:, None])
        np.add.at(dx, t, dh @ wi[e].T)
    return dict(dx=dx, dwi=dwi, dwo=dwo, dtopk_w=dw.reshape(T, k))


@pytest.mark.parametrize("T,emb,mlp,E,k", SHAPES)
def test_backward_from_the_8_bit_set(T, emb, mlp, E, k):
    d = _case(T, emb, mlp, E, k, T + 1)
    idx, w = moe.route(k, d["x"], d["wr"])
    _, saved = moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, save="int8")
    g = moe.ffn_bwd_ckpt(d["dy"], saved, d["wi"], d["wo"])
    ref = _bwd_ref(d, saved, k)
    for n in ref:
        got = g[n].float().cpu().double().numpy()
        assert np.isfinite(got).all(), n
        assert errors(got, ref[n])[0] <= REL, (n, errors(got, ref[n]))
    off = saved["group_offsets"].cpu().numpy()
    for e in np.nonzero(np.diff(off) == 0)[0]:
        assert (g["dwi"][e] == 0).all() and (g["dwo"][e] == 0).all()
    for need in (("dx",), ("dwi",), ("dwo",), ("dtopk_w",), ("dwi", "dx")):  # each alone: the same bits
        part = moe.ffn_bwd_ckpt(d["dy"], saved, d["wi"], d["wo"], need=need)
        assert set(part) == set(need)
        for n in need:
            assert _same_bits(part[n], g[n]), (need, n)


def test_gradients_stay_near_those_of_the_full_set():
    """The 8-bit set moves h and x by a uniform rounding of step 2^-6 of a block's largest power of two. 32 normal
    values reach 1 to 4 standard deviations, so the step is at most 4/64 and its error at most 4/64/sqrt(12) = 1.8 %
    of a standard deviation; a gradient takes two such values and bf16 roundings: below 5 %."""
    T, emb, mlp, E, k = 1000, 256, 320, 12, 3
    d = _case(T, emb, mlp, E, k, 5)
    idx, w = moe.route(k, d["x"], d["wr"])
    _, full = moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, save="full")
    _, int8 = moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, save="int8")
    a = moe.ffn_bwd(d["dy"], full, d["wi"], d["wo"], k)
    b = moe.ffn_bwd_ckpt(d["dy"], int8, d["wi"], d["wo"])
    for n in a:
        assert errors(b[n].float().cpu().numpy(), a[n].float().cpu().numpy())[0] < 0.05, n
    held = sum(int8[n].numel() * int8[n].element_size() for n in ("x_codes", "x_scales", "h_codes", "h_scales"))
    assert held == (T * emb + T * k * 2 * mlp) * 33 // 32


def _train(d, x, dy, logits, bias, k, cfg):
    route = dict(score=cfg["score"], renorm=cfg["renorm"], scale=cfg["scale"])
    idx, w = moe.route_scored(k, logits, balance_bias=bias, n_group=cfg["n_group"], topk_group=cfg["topk_group"],
                              group_top=cfg["group_top"], **route)
    y, saved = moe.ffn_fwd_routed(x, d["wi"], d["wo"], idx, w, save="int8")
    g = moe.ffn_bwd_ckpt(dy, saved, d["wi"], d["wo"])
    dl = moe.route_scored_bwd(logits, idx, w, g["dtopk_w"], **route)
    return (y, g["dx"], g["dwi"], g["dwo"], g["dtopk_w"], dl), saved


CONFIGS = [dict(score="sigmoid", renorm=True, scale=2.5, n_group=4, topk_group=2, group_top=2),
           dict(score="softmax", renorm=False, scale=1.0, n_group=1, topk_group=1, group_top=1)]


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: c["score"])
def test_training_step(cfg):
    T, emb, mlp, E, k = 300, 192, 256, 16, 4
    d = _case(T, emb, mlp, E, k, 21)
    gen = torch.Generator().manual_seed(3)
    logits = torch.randn((T, E), generator=gen)
    logits[5] = -float("inf")  # a token of which nothing is routed: y and its gradients are 0
    bias = (torch.randn(E, generator=gen) * 0.05).to(DEV)
    (y, dx, dwi, dwo, dw, dl), saved = _train(d, d["x"], d["dy"], logits.to(DEV), bias, k, cfg)
    ri, rw = su.route_scored(logits.double().numpy(), bias.cpu().double().numpy(), k, **cfg)
    assert np.array_equal(saved["topk_idx"].cpu().numpy(), ri)
    assert np.allclose(saved["topk_w"].cpu().numpy(), rw, rtol=1e-6, atol=0)
    assert (y[5] == 0).all() and (dx[5] == 0).all() and (dl[5] == 0).all()
    # y from the definition in 64 bits
    x, wi, wo = (d[n].cpu().double().numpy() for n in ("x", "wi", "wo"))
    ref = np.zeros((T, emb))
    for t in range(T):
        for j in range(k):
            h = x[t] @ wi[ri[t, j]]
            ref[t] += rw[t, j] * ((h[:mlp] / (1 + np.exp(-h[:mlp])) * h[mlp:]) @ wo[ri[t, j]])
    assert errors(y.float().cpu().numpy(), ref)[0] <= REL
    r = _bwd_ref(d, saved, k)
    for n, got in (("dx", dx), ("dwi", dwi), ("dwo", dwo), ("dtopk_w", dw)):
        assert errors(got.float().cpu().numpy(), r[n])[0] <= REL, n
    # dlogits against differences of sum(dtopk_w * weights)
    on = (rw != 0).astype(np.float64)
    ln = np.where(np.isfinite(logits.numpy()), logits.double().numpy(), 0.0)
    g = dw.cpu().double().numpy()
    num = np.zeros((T, E))
    with np.errstate(invalid="ignore"):
        for e in range(E):
            step = np.zeros((T, E))
            step[:, e] = 1e-5
            num[:, e] = ((su.weights(ln + step, ri, on, cfg["score"], cfg["renorm"], cfg["scale"]) -
                          su.weights(ln - step, ri, on, cfg["score"], cfg["renorm"], cfg["scale"])) * g).sum(1) / 2e-5
    num[5] = 0.0
    assert np.abs(dl.cpu().numpy() - num).max() <= 1e-5 * max(1.0, np.abs(g).max())


def test_training_step_graph_replays_and_streams_equal_eager():
    T, emb, mlp, E, k = 260, 128, 192, 16, 4
    cfg = CONFIGS[0]
    d = _case(T, emb, mlp, E, k, 8)
    gen = torch.Generator().manual_seed(1)
    bias = (torch.randn(E, generator=gen) * 0.05).to(DEV)

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        return (torch.randn((T, emb), generator=g).to(torch.bfloat16).to(DEV),
                torch.randn((T, emb), generator=g).to(torch.bfloat16).to(DEV), torch.randn((T, E), generator=g).to(DEV))

    buf = inputs(0)
    _train(d, *buf, bias, k, cfg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = _train(d, *buf, bias, k, cfg)
    for rep in range(4):
        new = inputs(rep + 1)
        for b, n in zip(buf, new):
            b.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        ref, _ = _train(d, *new, bias, k, cfg)
        for a, b in zip(out, ref):
            assert _same_bits(a, b), rep
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        o1, _ = _train(d, *buf, bias, k, cfg)
    with torch.cuda.stream(s2):
        o2, _ = _train(d, *buf, bias, k, cfg)
    torch.cuda.synchronize()
    for a, b, r in zip(o1, o2, ref):
        assert _same_bits(a, r) and _same_bits(b, r)


def test_no_tokens():
    emb, mlp, E, k = 64, 64, 4, 2
    d = _case(1, emb, mlp, E, k, 1)
    x = torch.empty((0, emb), dtype=torch.bfloat16, device=DEV)
    idx, w = moe.route_scored(k, torch.empty((0, E), device=DEV))
    for save in (None, "full", "int8"):
        y, saved = moe.ffn_fwd_routed(x, d["wi"], d["wo"], idx, w, save=save)
        assert y.shape == (0, emb)
    g = moe.ffn_bwd_ckpt(x, saved, d["wi"], d["wo"])
    assert g["dx"].shape == (0, emb) and (g["dwi"] == 0).all() and (g["dwo"] == 0).all()


def test_refused_arguments():
    d = _case(8, 64, 64, 4, 2, 1)
    idx, w = moe.route(2, d["x"], d["wr"])
    with pytest.raises(ValueError, match="save"):
        moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, save="fp8")
    with pytest.raises(ValueError):
        moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx[:4], w[:4])
    with pytest.raises(ValueError):
        moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"][:2], idx, w)
    with pytest.raises(TypeError):
        moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx.long(), w)
    with pytest.raises(moe.MoeError) as ei:
        moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert ei.value.status == moe._lib.MOE_ERR_WORKSPACE
    _, saved = moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, save="int8")
    with pytest.raises(ValueError):
        moe.ffn_bwd_ckpt(d["dy"][:4], saved, d["wi"], d["wo"])
    n = moe.workspace_bytes_routed(8, 64, 64, 4, 2, backward=True)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    a = moe.ffn_bwd_ckpt(d["dy"], saved, d["wi"], d["wo"], workspace=ws)
    b = moe.ffn_bwd_ckpt(d["dy"], saved, d["wi"], d["wo"])
    for k_ in a:
        assert _same_bits(a[k_], b[k_])


def test_bad_routings_stay_inside_the_buffers():
    """Expert ids out of range and the same expert twice: unspecified results, every write inside the outputs."""
    T, emb, mlp, E, k = 40, 64, 64, 4, 2
    d = _case(T, emb, mlp, E, k, 2)
    idx, w = moe.route(k, d["x"], d["wr"])
    idx[3] = torch.tensor([-1, 2**31 - 1], dtype=torch.int32)
    idx[7] = torch.tensor([1, 1], dtype=torch.int32)
    guard = torch.full((1 << 16,), 0x5a, dtype=torch.uint8, device=DEV)
    y, saved = moe.ffn_fwd_routed(d["x"], d["wi"], d["wo"], idx, w, save="int8")
    moe.ffn_bwd_ckpt(d["dy"], saved, d["wi"], d["wo"])
    torch.cuda.synchronize()
    assert (guard == 0x5a).all()


def test_bad_routings_leave_neighbouring_memory():
    """The same routings and an index set written over by hand, every output and scratch in a larger buffer."""
    import ctypes as C

    from mixture_experts_ffn_group_amd import _lib

    T, emb, mlp, E, k = 40, 64, 64, 4, 2
    S = T * k
    d = _case(T, emb, mlp, E, k, 2)
    idx, w = moe.route(k, d["x"], d["wr"])
    idx[3] = torch.tensor([-1, 2**31 - 1], dtype=torch.int32)
    idx[7] = torch.tensor([1, 1], dtype=torch.int32)
    guards = []

    def buf(n):
        b = torch.full((n + 8192,), 0x5a, dtype=torch.uint8, device=DEV)
        guards.append((b, n))
        return b[4096:4096 + n]

    sizes = dict(group_sizes=4 * E, group_offsets=4 * (E + 1), sorted_slot=4 * S, slot_row=4 * S, x_codes=T * emb,
                 x_scales=T * emb // 32, h_codes=S * 2 * mlp, h_scales=S * mlp // 16)
    saved = {n: buf(v) for n, v in sizes.items()}
    y = buf(T * emb * 2)
    out = [buf(n) for n in (T * emb * 2, E * emb * 2 * mlp * 2, E * mlp * emb * 2, S * 4)]
    s = _lib.shape(T, emb, mlp, E, k)
    wf, wb = moe.workspace_bytes_routed(T, emb, mlp, E, k), moe.workspace_bytes_routed(T, emb, mlp, E, k, True)
    ws_f, ws_b = buf(wf), buf(wb)
    s8 = _lib.MoeSaved8(*[saved[n].data_ptr() for n in sizes])
    dev = torch.device(DEV)
    moe._call("moe_ffn_fwd_routed", dev, C.byref(s), d["x"], idx, w, d["wi"], d["wo"], y, None, C.byref(s8), ws_f, wf)
    for offsets in (None, [0, 70, 20, 2**31 - 1, -5]):
        if offsets:
            saved["group_offsets"].view(torch.int32).copy_(torch.tensor(offsets, dtype=torch.int32))
            for n in ("sorted_slot", "slot_row"):
                saved[n].view(torch.int32)[::3] = 2**31 - 1
                saved[n].view(torch.int32)[1::3] = -7
        moe._call("moe_ffn_bwd_ckpt", dev, C.byref(s), d["dy"], w, C.byref(s8), d["wi"], d["wo"], *out, ws_b, wb)
    torch.cuda.synchronize()
    for b, n in guards:
        assert (b[:4096] == 0x5a).all() and (b[4096 + n:] == 0x5a).all()
