"""Plain 64-bit implementations of routing by scores and of the 8-bit checkpoint format, for the tests."""
import numpy as np


def route_scored(logits, bias, k, score, n_group, topk_group, group_top, renorm, scale):
    """(idx [T, k], w [T, k] float64) of logits [T, E] float64; bias [E] float64 or None."""
    T, E = logits.shape
    gs = E // n_group
    idx = np.zeros((T, k), np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        l = logits[t]
        on = ~np.isnan(l) & (l != -np.inf)
        s = np.zeros(E)
        if on.any():
            if score == "softmax":
                m = l[on].max()
                with np.errstate(invalid="ignore"):
                    s[on] = np.where(l[on] == m, 1.0, np.exp(np.minimum(l[on] - m, 0.0)))
                s[on] /= s[on].sum()
            else:
                with np.errstate(over="ignore"):
                    s[on] = 1.0 / (1.0 + np.exp(-l[on]))
        c = s.copy()
        if bias is not None:
            on &= ~np.isnan(bias) & (bias != -np.inf)
            c = c + bias
        rank = [(c[e] if bias is not None else l[e]) if on[e] else -np.inf for e in range(E)]
        kept = set(range(n_group))
        if topk_group < n_group:
            value = []
            for g in range(n_group):
                members = [e for e in range(g * gs, (g + 1) * gs) if on[e]]
                best = sorted(members, key=lambda e: (-rank[e], e))[:group_top]
                if not best:
                    value.append(-np.inf)
                elif group_top == 1:
                    value.append(rank[best[0]])
                else:
                    value.append(sum(sorted((c[e] for e in members), reverse=True)[:2]))
            kept = set(sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group])
        ok = [on[e] and e // gs in kept for e in range(E)]
        order = sorted(range(E), key=lambda e: (not ok[e], -rank[e] if ok[e] else 0.0, e))[:k]
        v = np.array([s[e] if ok[e] else 0.0 for e in order])
        if renorm:
            v = v / v.sum() if v.sum() > 0 else 0 * v
        idx[t], w[t] = order, v * scale
    return idx, w


def weights(logits, idx, on, score, renorm, scale):
    """The weights of given picks as a function of the logits (on [T, k]: picks that count)."""
    if score == "softmax":
        m = logits.max(axis=1, keepdims=True)
        s = np.exp(logits - m)
        s = s / s.sum(axis=1, keepdims=True)
    else:
        s = 1.0 / (1.0 + np.exp(-logits))
    v = np.take_along_axis(s, idx, axis=1) * on
    if renorm:
        v = v / v.sum(axis=1, keepdims=True)
    return v * scale


def ckpt_quantize(v):
    """codes [M, K] int8, scales [M, K/32] uint8 of v [M, K] float64 (values of fp32 or bf16)."""
    M, K = v.shape
    b = v.reshape(M, K // 32, 32)
    codes = np.zeros(b.shape, np.int8)
    scales = np.zeros(b.shape[:2], np.uint8)
    finite = np.isfinite(b).all(axis=2)
    amax = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(axis=2), 0.0)
    ex = np.frexp(amax)[1] - 1
    c = np.clip(np.where(amax > 0, ex + 127, 1), 1, 254)
    q = np.clip(np.rint(np.ldexp(np.where(finite[:, :, None], b, 0.0), 133 - c[:, :, None])), -127, 127)
    codes[:] = q
    scales[:] = np.where(finite, c, 255)
    return codes.reshape(M, K), scales


def ckpt_values(codes, scales):
    step = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 133))
    return codes.astype(np.float64) * np.repeat(step, 32, axis=1)
