"""Routing by scores and its gradient on the GPU against plain 64-bit implementations.

Tolerances. Picks are integers and must be equal; random fp32 logits put no two choice values within the 64-bit
rounding of each other, and ties are made on purpose with equal inputs. A weight is rounded once to fp32 from a
value good to a few 2^-24: |w - ref| <= 4 * 2^-24 * ref. A gradient sums at most k + 2 fp32 products of rounded
factors: its error is at most (k + 16) * 2^-24 of the sum of their magnitudes (8 of the 16 for the rounded argument of
the softmax's exponential, at logits within 16 of the largest), plus half a step of a bf16 output.
"""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_group_amd as moe
import scored_util as su

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _logits(T, E, seed, bf16=False, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) * spread
    return l.to(torch.bfloat16) if bf16 else l


def _check(l, bias, k, **cfg):
    cfg = dict(dict(score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0), **cfg)
    idx, w = moe.route_scored(k, l.to(DEV), balance_bias=None if bias is None else bias.to(DEV), **cfg)
    ri, rw = su.route_scored(l.double().numpy(), None if bias is None else bias.double().numpy(), k, **cfg)
    idx, w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    bad = np.nonzero((idx != ri).any(axis=1))[0]
    assert bad.size == 0, f"token {bad[:3]}: {idx[bad[:3]]} != {ri[bad[:3]]}"
    assert np.isfinite(w).all()
    assert (np.abs(w - rw) <= 4 * 2.0 ** -24 * rw + 1e-44).all(), np.abs(w - rw).max()
    return idx, w


CONFIGS = [
    dict(score="softmax", renorm=True),
    dict(score="softmax", renorm=False, scale=2.5),
    dict(score="sigmoid", renorm=True, scale=2.5),
    dict(score="sigmoid", renorm=False),
]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 37, 5), (64, 64, 8), (257, 60, 4), (130, 128, 8),
                                   (100, 256, 8), (33, 200, 17), (20, 256, 64), (9, 64, 64), (5, 3, 3)])
@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"{c['score']}-{'renorm' if c['renorm'] else 'raw'}")
@pytest.mark.parametrize("biased", [False, True])
def test_route_scored(T, E, k, cfg, biased):
    g = torch.Generator().manual_seed(E)
    bias = torch.randn(E, generator=g) * 0.05 if biased else None
    _check(_logits(T, E, T + E), bias, k, **cfg)


@pytest.mark.parametrize("E,n_group,topk_group,k", [(256, 8, 4, 8), (256, 16, 1, 16), (64, 8, 3, 6), (60, 10, 2, 7),
                                                    (128, 64, 9, 8), (256, 128, 40, 20), (8, 4, 4, 3), (96, 2, 1, 48)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_scored_groups(E, n_group, topk_group, k, group_top, score, biased):
    g = torch.Generator().manual_seed(E + n_group)
    bias = torch.randn(E, generator=g) * 0.1 if biased else None
    for T, bf16 in ((70, False), (5, True)):
        l = _logits(T, E, T + k)
        if bf16:  # distinct bf16 logits a row, so that group sums of two scores have no exact ties of unlike terms
            l = torch.stack([torch.randperm(E, generator=g).float() / 64 - 1 for _ in range(T)]).to(torch.bfloat16)
            if not biased and group_top == 2:
                continue  # permuted grids make equal sums from unlike pairs
        _check(l, bias, k, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top,
               renorm=True, scale=2.5)


@pytest.mark.parametrize("T,E,k", [(130, 128, 24), (50, 37, 20), (41, 256, 32), (33, 64, 17), (21, 160, 31)])
@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"{c['score']}-{'renorm' if c['renorm'] else 'raw'}")
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_scored_17_to_32_picks(T, E, k, cfg, biased, bf16):
    g = torch.Generator().manual_seed(E)
    bias = torch.randn(E, generator=g) * 0.05 if biased else None
    l = _logits(T, E, T + E, bf16)
    _check(l, bias, k, **cfg)
    l[3] = -float("inf")
    l[5, ::2] = float("nan")
    l[6, :] = 0.5
    _check(l, bias, k, **cfg)


@pytest.mark.parametrize("E,n_group,topk_group,k", [(256, 8, 4, 24), (96, 4, 2, 32), (200, 5, 3, 20), (256, 16, 2, 32)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_of_17_to_32_picks(E, n_group, topk_group, k, group_top, score, biased):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.1 if biased else None
    _check(_logits(70, E, 70 + k), bias, k, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)


def test_group_of_one_expert():
    _check(_logits(50, 32, 3), None, 5, score="sigmoid", n_group=32, topk_group=9, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_group,topk_group,group_top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_ties_go_to_the_lower_id(score, n_group, topk_group, group_top):
    T, E, k = 40, 64, 6
    g = torch.Generator().manual_seed(5)
    row = (torch.randint(0, 2, (T, E), generator=g)).float()  # two values only
    row[0] = 0.0
    bias = torch.zeros(E)
    bias[::2] = 0.25
    for b in (None, torch.zeros(E), bias):
        _check(row, b, k, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)


def test_signed_zeros_are_equal():
    l = torch.zeros(2, 16)
    l[0, ::2] = -0.0
    l[1, 1::2] = -0.0
    _check(l, None, 4)
    _check(l, None, 4, n_group=4, topk_group=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_group,topk_group,group_top", [(1, 1, 1), (8, 2, 1), (8, 2, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_disabled_experts_and_empty_rows(score, n_group, topk_group, group_top, renorm):
    T, E, k = 24, 64, 8
    l = _logits(T, E, 9)
    inf = float("inf")
    l[0] = -inf                        # nothing enabled: the lowest ids, weight 0
    l[1, 1:] = -inf                    # one enabled
    l[2, 5:] = -inf                    # fewer than k enabled
    l[3, ::2] = -inf
    l[4, 7] = float("nan")
    l[5] = float("nan")
    l[6] = torch.finfo(torch.float32).min   # a mask of the type's lowest value: enabled, and all equal
    l[7, 8:] = torch.finfo(torch.float32).min
    l[8, 3] = inf                      # +inf takes the softmax's whole mass
    l[9, 3] = l[9, 60] = inf
    l[10] = 100.0 * l[10]
    l[11] = -80.0
    bias = torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.1
    cfg = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top, renorm=renorm)
    _check(l, None, k, **cfg)
    _check(l, bias, k, **cfg)
    bias[40:] = -inf
    bias[3] = float("nan")
    _check(l, bias, k, **cfg)
    idx, w = _check(l, torch.full((E,), -inf), k, **cfg)
    assert (w == 0).all() and (idx == np.arange(k)).all()


def test_large_biases_and_close_scores():
    """Choice values that 32 bits cannot tell apart: scores next to each other under a large bias, and
    neighbouring fp32 logits."""
    T, E, k = 64, 128, 8
    l = _logits(T, E, 2)
    for b in (1.0, 1000.0, 1e6):
        _check(l, torch.full((E,), b), k, score="sigmoid")
        _check(l, torch.full((E,), -b), k, score="softmax", n_group=8, topk_group=3, group_top=2)
    base = _logits(T, 1, 3)
    near = (base.view(torch.int32) + torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))
                                                   for i in range(T)]).to(torch.int32)).view(torch.float32)
    for score in ("softmax", "sigmoid"):
        _check(near, torch.zeros(E), k, score=score)
        _check(near, None, k, score=score, n_group=4, topk_group=2, group_top=1)


def test_saturated_sigmoids_order_by_logit_without_a_bias():
    l = torch.arange(64).float().flip(0)[None, :] * 2 + 30  # all scores 1.0 in fp32
    _check(l, None, 8, score="sigmoid")
    _check(l.flip(1).contiguous(), None, 8, score="sigmoid", n_group=8, topk_group=2, group_top=1)


@pytest.mark.parametrize("T", [8191, 20000])
def test_many_tokens_match_the_64_bit_choice(T):
    """Enough tokens that some have neighbouring choice values within fp32 rounding."""
    g = torch.Generator().manual_seed(T)
    l = torch.randn((T, 256), generator=g)
    b = torch.randn(256, generator=g) * 0.05
    idx, w = moe.route_scored(8, l.to(DEV), balance_bias=b.to(DEV), score="sigmoid", n_group=8, topk_group=4,
                              group_top=2, scale=2.5)
    c = torch.sigmoid(l.double()) + b.double()
    gv = c.view(T, 8, 32).topk(2, dim=2).values.sum(2)
    keep = torch.zeros(T, 8, dtype=torch.bool).scatter_(1, gv.topk(4, dim=1).indices, True)
    c = c.masked_fill(~keep.repeat_interleave(32, 1), float("-inf"))
    assert torch.equal(idx.cpu().long(), c.topk(8, dim=1).indices)
    s = torch.sigmoid(l.double()).gather(1, idx.cpu().long())
    ref = 2.5 * s / s.sum(1, keepdim=True)
    assert ((w.cpu().double() - ref).abs() <= 4 * 2.0 ** -24 * ref).all()


@pytest.mark.parametrize("spread", [0.05, 0.002, 1e-5])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("E", [256, 100])
def test_many_tokens_of_softmax_scores_match_the_64_bit_choice(spread, grouped, E):
    """Biases down to the distance of neighbouring scores: most tokens then have close choice values."""
    T, k, G, kept = 8191, 7, 4, 2
    g = torch.Generator().manual_seed(E)
    l = torch.randn((T, E), generator=g)
    b = torch.randn(E, generator=g) * spread
    cfg = dict(n_group=G, topk_group=kept, group_top=2) if grouped else {}
    idx, w = moe.route_scored(k, l.to(DEV), balance_bias=b.to(DEV), score="softmax", renorm=False, **cfg)
    s = torch.softmax(l.double(), dim=1)
    c = s + b.double()
    if grouped:
        gv = c.view(T, G, E // G).topk(2, dim=2).values.sum(2)
        keep = torch.zeros(T, G, dtype=torch.bool).scatter_(1, gv.topk(kept, dim=1).indices, True)
        c = c.masked_fill(~keep.repeat_interleave(E // G, 1), float("-inf"))
    assert torch.equal(idx.cpu().long(), c.topk(k, dim=1).indices)
    ref = s.gather(1, idx.cpu().long())
    assert ((w.cpu().double() - ref).abs() <= 4 * 2.0 ** -24 * ref).all()


@pytest.mark.parametrize("k", [17, 32])
def test_many_tokens_and_picks_match_the_64_bit_choice(k):
    T = 8191
    g = torch.Generator().manual_seed(k)
    l = torch.randn((T, 256), generator=g)
    b = torch.randn(256, generator=g) * 0.05
    idx, w = moe.route_scored(k, l.to(DEV), balance_bias=b.to(DEV), score="sigmoid")
    c = torch.sigmoid(l.double()) + b.double()
    assert torch.equal(idx.cpu().long(), c.topk(k, dim=1).indices)
    s = torch.sigmoid(l.double()).gather(1, idx.cpu().long())
    ref = s / s.sum(1, keepdim=True)
    assert ((w.cpu().double() - ref).abs() <= 4 * 2.0 ** -24 * ref).all()


# ------------------------------------------------------------------ gradient

def _bwd_ref(l, idx, w, g, score, renorm, scale):
    """dlogits and the sum of magnitudes of the terms of each, from the formula in 64 bits."""
    T, E = l.shape
    m = np.where(np.isfinite(l), l, -np.inf).max(axis=1, keepdims=True)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax":
            s = np.exp(l - m)
            s = np.where(np.isfinite(l), s, 0.0)
            s = s / np.maximum(s.sum(axis=1, keepdims=True), 1e-300)
        else:
            s = 1.0 / (1.0 + np.exp(-l))
    on = w != 0
    wg = np.where(on, w * np.where(on, g, 0.0), 0.0)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    D = wg.sum(axis=1, keepdims=True)
    Da = np.abs(wg).sum(axis=1, keepdims=True)
    dl = wg - w * D / scale if renorm else wg
    ma = np.abs(wg) + w * Da / scale if renorm else np.abs(wg)
    if score == "sigmoid":
        f = 1.0 - np.take_along_axis(s, idx, axis=1)
        dl, ma = dl * f, ma * f
    np.put_along_axis(d, idx, np.where(on, dl, 0.0), axis=1)
    np.put_along_axis(mag, idx, np.where(on, ma, 0.0), axis=1)
    if score == "softmax" and not renorm:
        d, mag = d - s * D, mag + s * Da
    return d, mag


def _check_bwd(l, k, score, renorm, scale, seed, bias=None):
    idx, w = moe.route_scored(k, l.to(DEV), balance_bias=None if bias is None else bias.to(DEV), score=score,
                              renorm=renorm, scale=scale)
    g = torch.randn(idx.shape, generator=torch.Generator().manual_seed(seed))
    d = moe.route_scored_bwd(l.to(DEV), idx, w, g.to(DEV), score=score, renorm=renorm, scale=scale)
    assert d.dtype == l.dtype and d.shape == l.shape
    ref, mag = _bwd_ref(l.double().numpy(), idx.cpu().numpy().astype(np.int64), w.cpu().double().numpy(),
                        g.double().numpy(), score, renorm, scale)
    tol = (k + 16) * 2.0 ** -24 * mag + 1e-37
    if l.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    err = np.abs(d.cpu().double().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()
    return d


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (65, 37, 5), (130, 128, 8), (50, 256, 64), (31, 200, 1),
                                   (1000, 60, 4), (7, 64, 64)])
@pytest.mark.parametrize("score,renorm,scale", [("softmax", True, 1.0), ("softmax", False, 2.5),
                                                ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_scored_bwd(T, E, k, score, renorm, scale, bf16):
    _check_bwd(_logits(T, E, T, bf16), k, score, renorm, scale, seed=T + 1)


@pytest.mark.parametrize("T,E,k", [(130, 128, 24), (35, 37, 20), (50, 256, 32), (33, 60, 17)])
@pytest.mark.parametrize("score,renorm,scale", [("softmax", True, 1.0), ("softmax", False, 2.5),
                                                ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_scored_bwd_17_to_32_picks(T, E, k, score, renorm, scale, bf16):
    l = _logits(T, E, T, bf16)
    _check_bwd(l, k, score, renorm, scale, seed=T + 1)
    l[2, 5:] = -float("inf")  # fewer enabled than picks
    _check_bwd(l, k, score, renorm, scale, seed=T + 1)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_scored_bwd_disabled_picks_take_no_part(score, renorm):
    T, E, k = 12, 32, 6
    l = _logits(T, E, 4)
    inf = float("inf")
    l[0] = -inf
    l[1, 3:] = -inf
    l[2, ::2] = -inf
    bias = torch.zeros(E)
    bias[28:] = -inf
    d = _check_bwd(l, k, score, renorm, 1.0, 3, bias)
    assert (d[0] == 0).all()
    # a pick of weight 0 ignores its incoming gradient, whatever it is
    idx, w = moe.route_scored(k, l.to(DEV), score=score, renorm=renorm)
    g = torch.ones(T, k)
    g[0] = float("nan")
    d = moe.route_scored_bwd(l.to(DEV), idx, w, g.to(DEV), score=score, renorm=renorm)
    assert (d[0] == 0).all()


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_scored_bwd_against_differences(score, renorm):
    """Central differences of sum(g w) in 64 bits: step 1e-5, truncation about 1e-10, fp32 result 1e-6."""
    T, E, k, scale = 4, 12, 3, 2.5
    l = _logits(T, E, 8)
    idx, w = moe.route_scored(k, l.to(DEV), score=score, renorm=renorm, scale=scale)
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(2))
    d = moe.route_scored_bwd(l.to(DEV), idx, w, g.to(DEV), score=score, renorm=renorm, scale=scale).cpu().numpy()
    i = idx.cpu().numpy().astype(np.int64)
    ln, gn, on = l.double().numpy(), g.double().numpy(), np.ones((T, k))
    num = np.zeros((T, E))
    for e in range(E):
        h = np.zeros((T, E))
        h[:, e] = 1e-5
        num[:, e] = ((su.weights(ln + h, i, on, score, renorm, scale) -
                      su.weights(ln - h, i, on, score, renorm, scale)) * gn).sum(axis=1) / 2e-5
    assert np.abs(d - num).max() < 2e-6


def test_arguments_held_in_tensors_are_read_at_each_call():
    """k and scale as 0-dim tensors that change between the calls."""
    logits = torch.randn((5, 16), generator=torch.Generator().manual_seed(2)).to(DEV)
    k, scale = torch.tensor(4), torch.tensor(2.0)
    i4, w4 = moe.route_scored(k, logits, scale=scale)
    k.fill_(2)
    scale.fill_(1.0)
    i2, w2 = moe.route_scored(k, logits, scale=scale)
    ri, rw = moe.route_scored(2, logits)
    assert i4.shape == (5, 4) and torch.equal(i2, ri) and torch.equal(w2, rw)
    d = moe.route_scored_bwd(logits, ri, rw, torch.ones_like(rw), score="sigmoid", renorm=False, scale=scale)
    scale.fill_(3.0)
    d3 = moe.route_scored_bwd(logits, ri, rw, torch.ones_like(rw), score="sigmoid", renorm=False, scale=scale)
    assert torch.equal(d, d3)  # the factor is in the weights


def test_no_tokens():
    l = torch.zeros((0, 16), device=DEV)
    idx, w = moe.route_scored(3, l)
    assert idx.shape == (0, 3) and w.shape == (0, 3)
    assert moe.route_scored_bwd(l, idx, w, w).shape == (0, 16)


def test_neighbouring_memory_is_left_alone():
    """Outputs written inside larger buffers: nothing past the last token changes."""
    import ctypes as C
    from mixture_experts_ffn_group_amd import _lib
    T, E, k = 13, 60, 5
    l = _logits(T, E, 1).to(DEV)
    idx = torch.full((T * k + 64,), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T * k + 64,), -7.0, device=DEV)
    d = torch.full((T * E + 64,), -7.0, device=DEV)
    s, r = _lib.shape(T, 64, 64, E, k), _lib.MoeRouter(0, 1, 1, 1, 0, 1.0)
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    st = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert _lib.lib().moe_route_scored(C.byref(s), C.byref(r), p(l), 0, None, p(idx), p(w), st) == 0
    assert _lib.lib().moe_route_scored_bwd(C.byref(s), C.byref(r), p(l), 0, p(idx), p(w), p(w), p(d), st) == 0
    torch.cuda.synchronize()
    assert (idx[T * k:] == -7).all() and (w[T * k:] == -7).all() and (d[T * E:] == -7).all()
    assert (idx[:T * k] >= 0).all()


def test_out_of_range_picks_stay_inside_the_buffers():
    l = _logits(4, 16, 1).to(DEV)
    idx = torch.tensor([[0, -5], [99, 3], [2**31 - 1, 1], [-2**31, 7]], dtype=torch.int32, device=DEV)
    w = torch.full((4, 2), 0.5, device=DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            moe.route_scored_bwd(l, idx, w, w, score=score, renorm=renorm)
    torch.cuda.synchronize()


def test_graph_replays_equal_eager():
    T, E, k = 300, 256, 8
    l = _logits(T, E, 1).to(DEV)
    b = (torch.randn(E, generator=torch.Generator().manual_seed(3)) * 0.05).to(DEV)
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(4)).to(DEV)
    cfg = dict(score="sigmoid", renorm=True, scale=2.5)

    def step(x):
        idx, w = moe.route_scored(k, x, balance_bias=b, n_group=8, topk_group=4, group_top=2, **cfg)
        return idx, w, moe.route_scored_bwd(x, idx, w, g, **cfg)

    step(l)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(l)
    for rep in range(4):
        x = _logits(T, E, 10 + rep).to(DEV)
        l.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for a, r in zip(out, step(x)):
            assert torch.equal(a, r), rep
