"""The score router's gradient with picks that take no part: expert ids out of range, and disabled picks (weight 0)
whose incoming gradient is NaN. Every element of dlogits is compared with a 64-bit reference in which those picks are
left out, and the bytes on both sides of dlogits have to stay as they were. k = 2, 20 and 40 take three kernels.

Tolerance as in the router's other gradient tests: fp32 arithmetic, (k + 16) * 2^-24 of the sum of the terms'
magnitudes, and half a step of a bf16 output (2^-8 of its value).
"""
import ctypes as C

import numpy as np
import pytest
import torch

from mixture_experts_ffn_group_amd import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAD = 4096


def _reference(l, idx, w, g, score, renorm, scale):
    """(dlogits, sum of its terms' magnitudes) over the picks with an id in [0, E) and a weight."""
    T, E = l.shape
    s = np.exp(l - l.max(axis=1, keepdims=True))
    s = s / s.sum(axis=1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-l))
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E and w[t, j] != 0]
        total, size = sum(w[t, j] * g[t, j] for j in on), sum(abs(w[t, j] * g[t, j]) for j in on)
        if score == "softmax" and not renorm:
            d[t], mag[t] = -s[t] * total, s[t] * size
        for j in on:
            e = idx[t, j]
            f = 1 - s[t, e] if score == "sigmoid" else 1.0
            d[t, e] += w[t, j] * (g[t, j] - (total / scale if renorm else 0.0)) * f
            mag[t, e] += w[t, j] * (abs(g[t, j]) + (size / scale if renorm else 0.0)) * f
    return d, mag


@pytest.mark.parametrize("k", [2, 20, 40])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
def test_bad_and_disabled_picks_take_no_part(k, score, renorm, bf16):
    T, E, scale = 37, 61, 2.5
    rng = np.random.default_rng(k)
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    l = l.to(torch.bfloat16) if bf16 else l
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    bad = rng.random((T, k)) < 0.2
    bad[0], bad[1] = True, False
    idx[bad] = rng.choice([-1, -5, E, E + 1, 63, 64, 99, 2 ** 31 - 1, -2 ** 31], bad.sum())
    off = rng.random((T, k)) < 0.2
    off[2], off[1] = True, False
    w[off] = 0.0
    g[off] = np.nan
    ref, mag = _reference(l.double().numpy(), idx, w.astype(np.float64), g.astype(np.float64), score, renorm, scale)
    assert np.isfinite(ref).all() and (ref[0] == 0).all() and (ref[2] == 0).all() and (ref[1] != 0).any()

    n = T * E * l.element_size()
    buf = torch.full((PAD + n + PAD,), 0x5a, dtype=torch.uint8, device=DEV)
    args = [torch.from_numpy(v).to(DEV) for v in (idx, w, g)]
    ld = l.to(DEV)
    s, r = _lib.shape(T, 64, 64, E, k), _lib.MoeRouter(int(score == "sigmoid"), 1, 1, 1, int(renorm), scale)
    st = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = [C.c_void_p(t.data_ptr()) for t in (ld, *args)]
    _lib.check(_lib.lib().moe_route_scored_bwd(C.byref(s), C.byref(r), p[0], int(bf16), *p[1:],
                                               C.c_void_p(buf.data_ptr() + PAD), st), "moe_route_scored_bwd")
    torch.cuda.synchronize()
    out = buf.cpu()
    assert (out[:PAD] == 0x5a).all() and (out[PAD + n:] == 0x5a).all()
    d = out[PAD:PAD + n].clone().view(l.dtype).view(T, E).double().numpy()
    tol = (k + 16) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0)
    assert (np.abs(d - ref) <= tol).all(), np.argwhere(~(np.abs(d - ref) <= tol))[:5]
