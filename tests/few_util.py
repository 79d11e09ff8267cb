"""Plain 64-bit forms of the few-token layer and of the norms around the layer, on the CPU in numpy, with bounds on
what a right kernel's arithmetic may leave.

bf16 outputs are off by half a step of their own rounding, 2^-8 of the value. Before it, sums are fp32: a sum of n
terms is off by at most n * 2^-24 of the sum of their magnitudes, whatever its order.
"""
import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32, relative
H = 2.0 ** -8   # half a step of bf16


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def route(x, wr, bias, k):
    """Picks and weights: the k largest logits, ties to the lower id, and their softmax. NaN counts as less than -inf;
    the weight of either is 0, but NaN where all logits are NaN."""
    with np.errstate(invalid="ignore"):
        l = x @ wr
        if bias is not None:
            l = l + bias
    # descending, NaN last, equal ones by id
    idx = np.stack([np.lexsort((np.arange(len(r)), -np.where(np.isnan(r), -np.inf, r), np.isnan(r))) for r in l])[:, :k]
    top = np.take_along_axis(np.where(np.isnan(l), -np.inf, l), idx, 1)
    lost = np.isnan(l).all(1, keepdims=True)
    first = np.where(np.isfinite(top[:, :1]), top[:, :1], 0)
    w = np.exp(top - first)
    s = w.sum(1, keepdims=True)
    return idx.astype(np.int32), np.where(lost, np.nan, np.where(s > 0, w / np.where(s > 0, s, 1), 0))


def few(x, wi, wo, idx, w):
    """(y, bound on |y_kernel - y|) for the routing idx, w; wi [E, emb, 2*mlp], wo [E, mlp, emb]."""
    T, emb = x.shape
    mlp = wo.shape[1]
    y, err = np.zeros((T, emb)), np.zeros((T, emb))
    for t in range(T):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            if not 0 <= e < wi.shape[0] or w[t, j] == 0:
                continue
            h = x[t] @ wi[e]
            dh = (emb + 16) * U * (np.abs(x[t]) @ np.abs(wi[e]))
            g, u, dg, du = h[:mlp], h[mlp:], dh[:mlp], dh[mlp:]
            s = g / (1 + np.exp(-g))
            a = s * u
            # |silu'| < 1.1; exp and reciprocal of fp32 to a few steps; a kept to 16 bits
            da = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du + np.abs(a) * (2.0 ** -16 + 2.0 ** -19)
            o = a @ wo[e]
            do = da @ np.abs(wo[e]) + (mlp + 16) * U * ((np.abs(a) + da) @ np.abs(wo[e]))
            y[t] += w[t, j] * o
            err[t] += np.abs(w[t, j]) * (do + (idx.shape[1] * (mlp // 64 + 1) + 16) * U * (np.abs(a) @ np.abs(wo[e])))
    return y, err + H * (np.abs(y) + err) + 2.0 ** -133


def rms(v, weight, offset, eps):
    r = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * r * (1 if weight is None else weight + offset), r


def norm_grad(d, v, weight, offset, eps):
    """(dv, dweight, magnitudes of dv's terms, of dweight's terms)."""
    _, r = rms(v, None, 0, eps)
    f = 1 if weight is None else weight + offset
    g, xh = d * f, v * r
    m = (g * xh).mean(1, keepdims=True)
    mag = r * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    return r * (g - xh * m), (d * xh).sum(0), mag, np.abs(d * xh).sum(0)
