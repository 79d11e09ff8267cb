"""The expert router and the 8-bit activation checkpoints: the cases they are timed on, with plain forms.

Every operator here works on one sparse-MoE layer (T tokens, E experts, k picks per token, emb model width,
mlp expert width, S = T * k routed rows):

* ``route``: scores (softmax or sigmoid), balance bias, expert groups, top-k, weights;
* ``route_bwd``: the gradient of the weights with respect to the logits;
* ``ckpt``: rows written as 8-bit checkpoints and read back;
* ``swiglu_bwd``: the SwiGLU backward from an 8-bit h, with the row scale and its gradient;
* ``wgrad``: the grouped weight gradient whose left operand is the 8-bit checkpoint of the token rows, read
  through the routing.

``run`` computes them in elementary torch operations, or, where ``own`` is true, by the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32  # elements of a row that share one scale


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of four sequences through a 256-expert router with groups: latency
        dict(name="route_decode", op="route", T=4, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, dtype="f32"),
        # one device's tokens of a 256-expert layer, group-limited and bias-balanced
        dict(name="route_groups", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, renorm=True, scale=2.5, dtype="f32"),
        # one device's tokens of a 128-expert layer, softmax over all experts, weights renormalised
        dict(name="route_softmax", op="route", T=32768, E=128, k=8, score="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, renorm=True, scale=1.0, dtype="f32"),
        # its training counterpart on the 256-expert layer: only the picked logits have a gradient
        dict(name="route_bwd_sigmoid", op="route_bwd", T=8192, E=256, k=8, score="sigmoid", renorm=True, scale=2.5,
             dtype="f32"),
        # plain softmax weights: every logit has a gradient; bf16 logits, odd sizes
        dict(name="route_bwd_softmax", op="route_bwd", T=32749, E=60, k=4, score="softmax", renorm=False, scale=1.0,
             dtype="bf16"),
        # token rows of a wide layer kept for the backward
        dict(name="ckpt_tokens", op="ckpt", M=8192, K=7168, dtype="bf16"),
        # gate/up values as the first product leaves them, in 32 bits
        dict(name="ckpt_hidden", op="ckpt", M=65536, K=1536, dtype="f32"),
        # a short, odd batch
        dict(name="swiglu_bwd_small", op="swiglu_bwd", T=103, k=5, mlp=256),
        # 32768 tokens of a 128-expert, top-8 layer
        dict(name="swiglu_bwd_large", op="swiglu_bwd", T=32768, k=8, mlp=768),
        # few rows an expert, one expert without rows
        dict(name="wgrad_small", op="wgrad", T=500, k=3, E=12, emb=256, n=384, skew=0.0),
        # a skewed load over 32 experts, one without rows
        dict(name="wgrad_skewed", op="wgrad", T=4096, k=4, E=32, emb=1024, n=1024, skew=1.1),
        # 32768 tokens of a 128-expert, top-8 layer: the gradient of the gate/up weight
        dict(name="wgrad_large", op="wgrad", T=32768, k=8, E=128, emb=2048, n=1536, skew=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "ckpt", "swiglu_bwd", "wgrad"])
    if op in ("route", "route_bwd"):
        # expert counts with the group counts that divide them, from a few experts to the most supported
        E, groups = rng.choice([(8, (1, 2)), (16, (1, 4)), (37, (1,)), (60, (1, 4, 10)), (64, (1, 8)), (96, (1, 4)),
                                (128, (1, 4, 8)), (160, (1, 8)), (200, (1, 5)), (256, (1, 4, 8, 16))])
        G = rng.choice(groups)
        kept = G if G == 1 else rng.randint(1, G)
        k = rng.randint(1, min(rng.choice([2, 8, 8, 24]), kept * (E // G)))
        c = dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]))
        if c["T"] * E > 32768 * 128:
            c["T"] = 32768 * 128 // E
        if op == "route":
            c.update(bias=rng.random() < 0.5, n_group=G, topk_group=kept, group_top=rng.choice([1, 2]))
        return c
    if op == "ckpt":
        K = BLOCK * _log_int(rng, 2, 224)
        return dict(op=op, M=_log_int(rng, 1, 65536 * 1536 // K), K=K, dtype=rng.choice(["bf16", "f32"]))
    if op == "swiglu_bwd":
        mlp = 64 * rng.randint(1, 32)
        k = rng.randint(1, 8)
        return dict(op=op, T=_log_int(rng, 1, min(32768, 262144 * 768 // (mlp * k))), k=k, mlp=mlp)
    E = rng.choice([1, 5, 8, 32, 61, 128])
    emb, n = 64 * rng.randint(1, 32), 128 * rng.randint(1, 12)
    k = rng.randint(1, min(E, 8))
    return dict(op=op, T=_log_int(rng, 1, 8192), k=k, E=E, emb=emb, n=n, skew=rng.choice([0.0, 1.1]))


def _route_flops(c):
    return c["T"] * c["E"] * 8  # an exponential, its sum, the bias, the comparison


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * c["E"] * size + c["T"] * c["k"] * 8 + (c["E"] * 4 if c["bias"] else 0),
                "flops": _route_flops(c)}
    if c["op"] == "route_bwd":
        size = 4 if c["dtype"] == "f32" else 2
        dense = c["score"] == "softmax" and not c["renorm"]
        read = c["T"] * c["E"] * size if dense else (c["T"] * c["k"] * size if c["score"] == "sigmoid" else 0)
        return {"bytes": read + c["T"] * c["E"] * size + c["T"] * c["k"] * 12,
                "flops": _route_flops(c) if dense else c["T"] * c["k"] * 12}
    if c["op"] == "ckpt":
        n = c["M"] * c["K"]
        held = n + n // BLOCK
        src = n * (2 if c["dtype"] == "bf16" else 4)
        return {"bytes": src + 2 * held + n * 2, "flops": 4 * n}  # read, held, held read, bf16 values
    if c["op"] == "swiglu_bwd":
        S, m = c["T"] * c["k"], c["mlp"]
        return {"bytes": S * m * 2 + S * 2 * m + S * 2 * m // BLOCK + S * 2 * m * 2 + S * m * 2 + S * 12,
                "flops": S * m * 16}
    S = c["T"] * c["k"]
    return {"bytes": c["T"] * c["emb"] + c["T"] * c["emb"] // BLOCK + S * c["n"] * 2 + S * 4 +
            c["E"] * c["emb"] * c["n"] * 2,
            "flops": 2 * S * c["emb"] * c["n"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _logits(case, g):
    l = _randn(g, case["T"], case["E"])  # N(0, 0.02) router weights on unit rows of 2048 columns: about 1
    return l.to(torch.bfloat16) if case["dtype"] == "bf16" else l


def _mx(v):
    """8-bit codes and block scales of the rows v (values held as integers times a power of two)."""
    M, K = v.shape
    b = v.float().view(M, K // BLOCK, BLOCK)
    ex = torch.frexp(b.abs().amax(dim=2))[1] - 1
    c = (ex + 127).clamp(1, 254)
    inv = ((1023 + 133 - c.long()) << 52).view(torch.float64)  # 2^(133 - c) from its bits
    code = torch.round(b.double() * inv[:, :, None]).clamp(-127, 127)
    return code.to(torch.int8).view(M, K), c.to(torch.uint8)


def _routing(T, E, k, skew, g, empty):
    """Distinct picks per token, Zipf-skewed if asked; `empty` leaves the last expert without rows."""
    score = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-20, 1 - 1e-7)))
    score = score - skew * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    if empty:
        score[:, E - 1] = -math.inf
    idx = torch.topk(score, k, dim=1).indices
    flat = idx.reshape(-1)
    slot = torch.sort(flat, stable=True).indices.to(torch.int32)
    sizes = torch.bincount(flat, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(sizes, 0).to(torch.int32)
    return slot, off


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "route":
        st["logits"] = _logits(case, g)
        # what a balance update leaves: small values of both signs
        st["bias"] = 0.05 * _randn(g, case["E"]) if case["bias"] else None
    elif case["op"] == "route_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = _logits(case, g)
        full = dict(case, bias=False, n_group=1, topk_group=1, group_top=1)
        st["idx"], st["w"] = _route(dict(case=full, logits=st["logits"], bias=None))
        st["g"] = _randn(g, T, k)
    elif case["op"] == "ckpt":
        v = _randn(g, case["M"], case["K"])
        v *= torch.exp(_randn(g, case["M"], 1))  # rows of unlike size
        st["src"] = v.to(torch.bfloat16) if case["dtype"] == "bf16" else v
    elif case["op"] == "swiglu_bwd":
        T, k, m = case["T"], case["k"], case["mlp"]
        S = T * k
        h = _randn(g, S, 2 * m)
        st["codes"], st["scales"] = [], []
        for i in range(0, S, 32768):
            cd, sc = _mx(h[i:i + 32768])
            st["codes"].append(cd)
            st["scales"].append(sc)
        st["codes"], st["scales"] = torch.cat(st["codes"]), torch.cat(st["scales"])
        st["da"] = (0.5 * _randn(g, S, m)).to(torch.bfloat16)
        st["slot"] = torch.randperm(S, generator=g, device=DEV).to(torch.int32)
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        st["w"] = (w / w.sum(1, keepdim=True)).reshape(-1).contiguous()
    else:
        T, k, E = case["T"], case["k"], case["E"]
        st["codes"], st["scales"] = _mx(_randn(g, T, case["emb"]))
        st["slot"], st["off"] = _routing(T, E, k, case["skew"], g, empty=k < E)
        st["host_off"] = st["off"].tolist()  # the plain form's loop over the experts
        st["D"] = (0.1 * _randn(g, T * k, case["n"])).to(torch.bfloat16)
    return st


# ------------------------------------------------------------------ plain forms

def _route(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    # which expert is picked hangs on neighbouring scores: in 64 bits
    l = st["logits"].double()
    s = torch.softmax(l, dim=1) if c["score"] == "softmax" else torch.sigmoid(l)
    choice = s if st["bias"] is None else s + st["bias"].double()
    order = l if st["bias"] is None else choice  # the scores rise with the logits
    if c["topk_group"] < G:
        key = order if c["group_top"] == 1 else choice
        top = torch.topk(key.view(T, G, E // G), c["group_top"], dim=2).values.sum(dim=2)
        kept = torch.sort(top, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        mask = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        order = order.masked_fill(~mask.repeat_interleave(E // G, dim=1), -math.inf)
    idx = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), (w * c["scale"]).float()


def _route_bwd(st):
    c = st["case"]
    l, g, w, idx = st["logits"].float(), st["g"], st["w"], st["idx"].long()
    if c["renorm"]:
        wg = w * (g - (w * g).sum(dim=1, keepdim=True) / c["scale"])
    else:
        wg = w * g
    d = torch.zeros_like(l)
    if c["score"] == "sigmoid":
        d.scatter_(1, idx, wg * torch.sigmoid(-l.gather(1, idx)))
    elif c["renorm"]:
        d.scatter_(1, idx, wg)
    else:
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        d = -(e / e.sum(dim=1, keepdim=True)) * wg.sum(dim=1, keepdim=True)
        d.scatter_add_(1, idx, wg)
    return d.to(st["logits"].dtype)


def _values(codes, scales):
    """fp32 values of 8-bit rows."""
    M, K = codes.shape
    step = (scales.int() << 23).view(torch.float32) / 64  # 2^(c - 127) from its bits, 2^-6 a unit of the code
    return (codes.view(M, K // BLOCK, BLOCK).float() * step[:, :, None]).view(M, K)


def _ckpt(st):
    codes, scales = _mx(st["src"])
    return _values(codes, scales).to(torch.bfloat16)


def _swiglu_bwd(st):
    m = st["case"]["mlp"]
    h = _values(st["codes"], st["scales"])
    g, u = h[:, :m], h[:, m:]
    slot = st["slot"].long()
    da = st["da"].float()
    s = torch.sigmoid(g)
    a = g * s * u
    dscale = torch.empty_like(st["w"])
    dscale[slot] = (da * a).sum(dim=1)
    da = da * st["w"][slot][:, None]
    dh = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], dim=1)
    return dh.to(torch.bfloat16), a.to(torch.bfloat16), dscale


def _wgrad(st):
    c = st["case"]
    x = _values(st["codes"], st["scales"])
    tok = (st["slot"] // c["k"]).long()
    out = torch.zeros((c["E"], c["emb"], c["n"]), dtype=torch.bfloat16, device=x.device)
    for e in range(c["E"]):
        lo, hi = st["host_off"][e], st["host_off"][e + 1]
        if hi > lo:
            out[e] = (x[tok[lo:hi]].t() @ st["D"][lo:hi].float()).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ the framework's calls

def _own(st):
    import mixture_experts_ffn_group_amd as moe
    c = st["case"]
    if c["op"] == "route":
        return moe.route_scored(c["k"], st["logits"], balance_bias=st["bias"], score=c["score"],
                                n_group=c["n_group"], topk_group=c["topk_group"], group_top=c["group_top"],
                                renorm=c["renorm"], scale=c["scale"])
    if c["op"] == "route_bwd":
        return moe.route_scored_bwd(st["logits"], st["idx"], st["w"], st["g"], score=c["score"], renorm=c["renorm"],
                                    scale=c["scale"])
    if c["op"] == "ckpt":
        codes, scales = moe.ckpt_quantize(st["src"])
        return moe.ckpt_dequantize(codes, scales)
    if c["op"] == "swiglu_bwd":
        return moe.swiglu_bwd_ckpt(st["da"], st["codes"], st["scales"], row_slot=st["slot"], slot_scale=st["w"])
    return moe.grouped_gemm_wgrad_ckpt(st["codes"], st["scales"], st["D"], st["off"], c["E"], row_slot=st["slot"],
                                       slot_div=c["k"])


_PLAIN = {"route": _route, "route_bwd": _route_bwd, "ckpt": _ckpt, "swiglu_bwd": _swiglu_bwd, "wgrad": _wgrad}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_route(c, st):
    l = st["logits"].double()
    T, E = l.shape
    if c["score"] == "softmax":
        s = torch.exp(l - torch.logsumexp(l, dim=1, keepdim=True))
    else:
        s = 1 / (1 + torch.exp(-l))
    value = s.clone() if st["bias"] is None else s + st["bias"].double()[None, :]
    rank = l.clone() if st["bias"] is None else value.clone()
    ids = torch.arange(E, device=l.device)
    G, gs = c["n_group"], E // c["n_group"]
    alive = torch.ones((T, E), dtype=torch.bool, device=l.device)
    if c["topk_group"] < G:
        gv = []
        for gi in range(G):
            part = (rank if c["group_top"] == 1 else value)[:, gi * gs:(gi + 1) * gs]
            best = part.amax(dim=1)
            if c["group_top"] == 2:
                first = torch.where(part == best[:, None], ids[:gs], E).amin(dim=1)
                best = best + part.masked_fill(ids[:gs] == first[:, None], -math.inf).amax(dim=1)
            gv.append(best)
        gv = torch.stack(gv, dim=1)
        alive[:] = False
        for _ in range(c["topk_group"]):
            m = gv.amax(dim=1, keepdim=True)
            pick = torch.where(gv == m, ids[:G], E).amin(dim=1)
            gv.scatter_(1, pick[:, None], -math.inf)
            alive |= (ids // gs) == pick[:, None]
    picks = []
    for _ in range(c["k"]):
        r = rank.masked_fill(~alive, -math.inf)
        p = torch.where(r == r.amax(dim=1, keepdim=True), ids, E).amin(dim=1)
        alive &= ids != p[:, None]
        picks.append(p)
    idx = torch.stack(picks, dim=1)
    w = torch.stack([s[torch.arange(T, device=l.device), p] for p in picks], dim=1)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), w * c["scale"]


def _exact_route_bwd(c, st):
    # from the scores: L = sum_j g_j w_j(s(l)), w the exact weights of the given picks
    l, g = st["logits"].double(), st["g"].double()
    idx = st["idx"].long()
    T, E = l.shape
    s = torch.softmax(l, dim=1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-l))
    sp = s.gather(1, idx)
    if c["renorm"]:
        tot = sp.sum(dim=1, keepdim=True)
        dsp = c["scale"] * (g / tot - (g * sp).sum(dim=1, keepdim=True) / tot ** 2)
    else:
        dsp = c["scale"] * g
    ds = torch.zeros_like(s).scatter_(1, idx, dsp)
    if c["score"] == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(dim=1, keepdim=True))


def _exact_values(codes, scales):
    step = torch.tensor([2.0 ** (c - 133) for c in range(256)], dtype=torch.float64, device=codes.device)
    return codes.double() * step[scales.long()].repeat_interleave(BLOCK, dim=1)


def _exact_ckpt(c, st):
    v = st["src"].double()
    M, K = v.shape
    out = torch.empty_like(v)
    for i in range(0, M, 8192):
        b = v[i:i + 8192].reshape(-1, BLOCK)
        top = b.abs().amax(dim=1, keepdim=True).clamp_min(2.0 ** -126)
        step = (top.view(torch.int64) & 0x7ff0000000000000).view(torch.float64) / 64  # 2^floor(log2 top) / 64
        out[i:i + 8192] = (torch.round(b / step).clamp(-127, 127) * step).view(-1, K)
    return out


def _exact_swiglu_bwd(c, st):
    m = c["mlp"]
    S = st["da"].shape[0]
    dh = torch.empty((S, 2 * m), dtype=torch.float64, device=DEV)
    a = torch.empty((S, m), dtype=torch.float64, device=DEV)
    dscale = torch.empty(S, dtype=torch.float64, device=DEV)
    for i in range(0, S, 32768):
        v = _exact_values(st["codes"][i:i + 32768], st["scales"][i:i + 32768])
        g, u = v.split(m, dim=1)
        e = torch.exp(-g)
        sl = st["slot"][i:i + 32768].long()
        w = st["w"].double()[sl].unsqueeze(1)
        da = st["da"][i:i + 32768].double()
        a[i:i + 32768] = g / (1 + e) * u
        dscale[sl] = (da * a[i:i + 32768]).sum(dim=1)
        dh[i:i + 32768, :m] = w * da * u * ((1 + e) + g * e) / (1 + e) ** 2
        dh[i:i + 32768, m:] = w * da * g / (1 + e)
    return dh, a, dscale


def _exact_wgrad(c, st):
    x = _exact_values(st["codes"], st["scales"])
    out = torch.zeros((c["E"], c["emb"], c["n"]), dtype=torch.float64, device=DEV)
    off = st["off"].cpu().numpy()
    for e in range(c["E"]):
        rows = slice(int(off[e]), int(off[e + 1]))
        tok = torch.div(st["slot"][rows], c["k"], rounding_mode="floor").long()
        out[e] = torch.mm(x.index_select(0, tok).t().contiguous(), st["D"][rows].double())
    return out


_EXACT = {"route": _exact_route, "route_bwd": _exact_route_bwd, "ckpt": _exact_ckpt,
          "swiglu_bwd": _exact_swiglu_bwd, "wgrad": _exact_wgrad}


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))
