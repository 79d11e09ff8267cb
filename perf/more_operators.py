"""The expert layer for a few tokens, and the norms around the layer: the cases they are timed on, with plain forms.

* ``few``: router, experts and combine of T <= 64 tokens, on bf16 weights;
* ``few_mx``: the same on MXFP8 weights (E4M3 codes, a power-of-two scale per 32 along the contraction);
* ``norm``: the RMS norm before the layer, forward or backward (with the residual's gradient added);
* ``block``: what follows the layer, forward or backward: its output (given, or combined from expert rows), the norm
  after it, a gate, the residual sum with its scales, and the next norm.

``run`` computes them in elementary torch operations, or, where ``own`` is true, by the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
MAX_T = 64      # most tokens of the few-token layer
MX_BLOCK = 32   # elements along the contraction that share one MXFP8 scale
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence's decode step through a 128-expert, top-8 layer: latency
        dict(name="few_one", op="few", T=1, emb=2048, mlp=768, E=128, k=8, bias=False, routed=False),
        # a few sequences, odd sizes, few experts, a biased router
        dict(name="few_odd", op="few", T=5, emb=1088, mlp=448, E=60, k=4, bias=True, routed=False),
        # four sequences through a wide 256-expert layer, routed by the caller
        dict(name="few_wide", op="few", T=4, emb=7168, mlp=2048, E=256, k=8, bias=False, routed=True),
        # a full decode batch: nearly every expert has tokens
        dict(name="few_batch", op="few", T=64, emb=2048, mlp=768, E=128, k=8, bias=False, routed=False),
        # two sequences on 8-bit weights
        dict(name="few_mx_two", op="few_mx", T=2, emb=2048, mlp=768, E=128, k=8, bias=False, routed=False),
        # a batch on 8-bit weights of the wide layer's sizes, an odd count
        dict(name="few_mx_batch", op="few_mx", T=19, emb=7168, mlp=2048, E=64, k=8, bias=True, routed=False),
        # the norm before the layer in a decode step
        dict(name="norm_decode", op="norm", way="fwd", T=4, emb=7168, xt="bf16", wt="f32", offset=0.0),
        # its gradient in training, the residual stream in 32 bits
        dict(name="norm_bwd", op="norm", way="bwd", T=8192, emb=7168, xt="f32", wt="f32", offset=0.0),
        # after the layer in a decode step: norm, gate per channel, residual, next norm
        dict(name="block_decode", op="block", way="fwd", T=3, emb=2048, xt="bf16", wt="bf16", offset=1.0, k=0, post=True,
             gate="channel", gt="f32", scale=1.0, res_scale=1.0, next=True),
        # after the layer in training: the same on a device's tokens
        dict(name="block_train", op="block", way="fwd", T=32768, emb=2048, xt="bf16", wt="bf16", offset=1.0, k=0,
             post=True, gate="channel", gt="f32", scale=0.5, res_scale=1.0, next=True),
        # serving a long prompt: the expert rows combined on the way, residual in 32 bits
        dict(name="block_rows", op="block", way="fwd", T=8192, emb=7168, xt="f32", wt="f32", offset=0.0, k=8, post=True,
             gate="none", gt="f32", scale=1.0, res_scale=1.0, next=True),
        # the gradient of all of it, a gate per token
        dict(name="block_bwd", op="block", way="bwd", T=32749, emb=2048, xt="bf16", wt="f32", offset=0.0, k=0,
             post=True, gate="token", gt="bf16", scale=0.5, res_scale=1.0, next=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "few_mx", "norm", "block", "block"])
    if op in ("few", "few_mx"):
        emb, mlp = 64 * _log_int(rng, 1, 112), 64 * _log_int(rng, 1, 32)
        E = rng.choice([1, 4, 8, 16, 37, 60, 64, 128, 160, 256])
        k = rng.randint(1, min(E, rng.choice([2, 8, 8, 16])))
        T = _log_int(rng, 1, MAX_T)
        # no more weights than the wide layer's, no more read than a batch of the 128-expert layer reads
        E = max(k, min(E, 256 * 7168 * 2048 // (emb * mlp)))
        while min(E, T * k) * emb * mlp > 128 * 2048 * 768 and T > 1:
            T -= 1
        return dict(op=op, T=T, emb=emb, mlp=mlp, E=E, k=k, bias=rng.random() < 0.3, routed=rng.random() < 0.4)
    emb = 64 * _log_int(rng, 2, 128)
    c = dict(op=op, way=rng.choice(["fwd", "bwd"]), emb=emb, xt=rng.choice(["bf16", "f32"]),
             wt=rng.choice(["bf16", "f32", "none"]), offset=rng.choice([0.0, 1.0]))
    c["T"] = _log_int(rng, 1, 32768 * 2048 // emb)
    if op == "norm":
        return c
    c.update(k=rng.choice([0, 0, 2, 8]) if c["way"] == "fwd" else 0, post=rng.random() < 0.75,
             gate=rng.choice(["none", "channel", "token", "full"]), gt=rng.choice(["bf16", "f32"]),
             scale=rng.choice([1.0, 0.5]), res_scale=rng.choice([1.0, 0.75]), next=rng.random() < 0.7)
    if c["k"]:
        c["T"] = max(1, min(c["T"], 8192 * 7168 // emb))
    return c


_SIZE = {"bf16": 2, "f32": 4, "none": 0}
_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def work(case):
    c = case
    T, emb = c["T"], c["emb"]
    if c["op"] in ("few", "few_mx"):
        mlp, E, k = c["mlp"], c["E"], c["k"]
        hit = E * (1 - (1 - k / E) ** T)  # experts with a token, expected
        per = 2.0 if c["op"] == "few" else 1 + 4 / 64
        nbytes = hit * 3 * emb * mlp * per + T * emb * 4 + T * k * 8
        flops = 6 * T * k * emb * mlp
        if not c["routed"]:
            nbytes += emb * E * 4
            flops += 2 * T * emb * E
        return {"bytes": nbytes, "flops": flops}
    n, xs, ws = T * emb, _SIZE[c["xt"]], _SIZE[c["wt"]]
    if c["op"] == "norm":
        if c["way"] == "fwd":
            return {"bytes": n * (xs + 2) + emb * ws, "flops": 4 * n}
        return {"bytes": n * (2 + 3 * xs) + emb * (ws + (4 if ws else 0)), "flops": 10 * n}
    g = {"none": 0, "channel": emb, "token": T, "full": n}[c["gate"]] * _SIZE[c["gt"]]
    if c["way"] == "fwd":
        src = n * 2 * c["k"] + T * c["k"] * 8 if c["k"] else n * 2
        return {"bytes": src + 2 * n * xs + g + (n * 2 if c["next"] else 0) + emb * ws * (c["post"] + c["next"]),
                "flops": n * (10 + 2 * c["k"])}
    gout = {"none": 0, "channel": 4 * emb, "token": 4 * T, "full": n * _SIZE[c["gt"]]}[c["gate"]]
    need_y = c["post"] or c["gate"] != "none"
    return {"bytes": n * (2 * xs + 2 + (2 if need_y else 0)) + (n * (2 + xs) if c["next"] else 0) + g + gout +
            emb * (ws + (4 if ws else 0)) * (c["post"] + c["next"]),
            "flops": 24 * n}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _mx(w):
    """MXFP8 of one expert's weight w [K, N]: codes [N, K] and scales [K/64, N, 4] (two used bytes a slice)."""
    K, N = w.shape
    b = w.float().t().contiguous().view(N, K // MX_BLOCK, MX_BLOCK)
    ex = torch.frexp(b.abs().amax(dim=2))[1] - 1
    c = (ex - 8 + 127).clamp(0, 254)
    v = torch.ldexp(b, (127 - c)[:, :, None]).clamp(-448, 448)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8).view(N, K)
    scales = torch.zeros((K // 64, N, 4), dtype=torch.uint8, device=w.device)
    scales[:, :, :2] = c.to(torch.uint8).view(N, K // 64, 2).permute(1, 0, 2)
    return codes, scales


def prepare(case, seed):
    c = case
    g = _gen(seed)
    st = dict(case=c)
    T, emb = c["T"], c["emb"]
    if c["op"] in ("few", "few_mx"):
        mlp, E, k = c["mlp"], c["E"], c["k"]
        st["x"] = _randn(g, T, emb).to(torch.bfloat16)
        # gate and up values of size about one whatever the widths
        sig_i, sig_o = 1 / math.sqrt(emb), 1 / math.sqrt(mlp)
        if c["op"] == "few":
            st["wi"] = torch.empty((E, emb, 2 * mlp), dtype=torch.bfloat16, device=DEV)
            st["wo"] = torch.empty((E, mlp, emb), dtype=torch.bfloat16, device=DEV)
        else:
            st["wq"] = dict(wi_codes=torch.empty((E, 2 * mlp, emb), dtype=torch.uint8, device=DEV),
                            wi_scales=torch.empty((E, emb // 64, 2 * mlp, 4), dtype=torch.uint8, device=DEV),
                            wo_codes=torch.empty((E, emb, mlp), dtype=torch.uint8, device=DEV),
                            wo_scales=torch.empty((E, mlp // 64, emb, 4), dtype=torch.uint8, device=DEV), mlp=mlp)
        for e in range(E):
            wi, wo = _randn(g, emb, 2 * mlp) * sig_i, _randn(g, mlp, emb) * sig_o
            if c["op"] == "few":
                st["wi"][e], st["wo"][e] = wi, wo
            else:
                st["wq"]["wi_codes"][e], st["wq"]["wi_scales"][e] = _mx(wi)
                st["wq"]["wo_codes"][e], st["wq"]["wo_scales"][e] = _mx(wo)
        st["wr"] = 0.02 * _randn(g, emb, E)
        st["bias"] = 0.1 * _randn(g, E) if c["bias"] else None
        if c["routed"]:
            st["idx"], st["w"] = _route(st)
        return st
    xt = _DTYPE[c["xt"]]

    def weight():
        if c["wt"] == "none":
            return None
        return ((1 - c["offset"]) + 0.1 * _randn(g, emb)).to(_DTYPE[c["wt"]])

    size = torch.exp(0.5 * _randn(g, T, 1))  # rows of unlike size
    if c["op"] == "norm":
        st["x"] = (_randn(g, T, emb) * size).to(xt)
        st["weight"] = weight()
        if c["way"] == "bwd":
            st["dy"] = _randn(g, T, emb).to(torch.bfloat16)
            st["dres"] = _randn(g, T, emb).to(xt)
        return st
    st["post_weight"] = weight() if c["post"] else None
    st["next_weight"] = weight() if c["next"] else None
    gate = {"none": None, "channel": (emb,), "token": (T, 1), "full": (T, emb)}[c["gate"]]
    st["gate"] = None if gate is None else (0.5 + 0.25 * _randn(g, *gate)).to(_DTYPE[c["gt"]])
    st["y"] = None
    if c["k"]:
        k = c["k"]
        st["ys"] = torch.empty((T * k, emb), dtype=torch.bfloat16, device=DEV)
        for i in range(0, T * k, 8192):
            st["ys"][i:i + 8192] = _randn(g, *st["ys"][i:i + 8192].shape)
        st["slot_row"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        st["topk_w"] = w / w.sum(dim=1, keepdim=True)
    else:
        st["y"] = (_randn(g, T, emb) * size).to(torch.bfloat16)
    st["res"] = _randn(g, T, emb).to(xt)  # the residual, or the stored sum in the backward
    if c["way"] == "bwd":
        st["dout"] = _randn(g, T, emb).to(xt)
        st["dnext"] = _randn(g, T, emb).to(torch.bfloat16) if c["next"] else None
    return st


# ------------------------------------------------------------------ plain forms

def _route(st):
    l = st["x"].double() @ st["wr"].double()  # the picks hang on neighbouring logits: in 64 bits
    if st["bias"] is not None:
        l = l + st["bias"].double()
    top, idx = torch.sort(l, dim=1, descending=True, stable=True)
    k = st["case"]["k"]
    e = torch.exp(top[:, :k] - top[:, :1])
    return idx[:, :k].to(torch.int32), (e / e.sum(dim=1, keepdim=True)).float()


def _mx_values(codes, scales):
    """fp32 values [n, K, N] of the chosen experts' codes [n, N, K] and scales [n, K/64, N, 4]."""
    n, N, K = codes.shape
    s = scales[..., :2].permute(0, 2, 1, 3).reshape(n, N, K // MX_BLOCK, 1)
    v = codes.view(torch.float8_e4m3fn).float().view(n, N, K // MX_BLOCK, MX_BLOCK)
    return torch.ldexp(v, s.int() - 127).view(n, N, K).transpose(1, 2).contiguous()


def _few(st):
    c = st["case"]
    mlp = c["mlp"]
    idx, w = (st["idx"], st["w"]) if c["routed"] else _route(st)
    y = torch.empty((c["T"], c["emb"]), dtype=torch.float32, device=DEV)
    for t in range(c["T"]):
        e = idx[t].long()
        if c["op"] == "few":
            wi, wo = st["wi"][e].float(), st["wo"][e].float()
        else:
            q = st["wq"]
            wi, wo = _mx_values(q["wi_codes"][e], q["wi_scales"][e]), _mx_values(q["wo_codes"][e], q["wo_scales"][e])
        h = torch.matmul(st["x"][t].float(), wi)
        a = h[:, :mlp] * torch.sigmoid(h[:, :mlp]) * h[:, mlp:]
        o = torch.bmm(a[:, None, :], wo)[:, 0]
        y[t] = (w[t][:, None] * o).sum(dim=0)
    y = y.to(torch.bfloat16)
    return y if c["routed"] else (y, idx, w)


def _rms(x):
    return torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)


def _scaled(x, weight, offset):
    return x if weight is None else x * (offset + weight.float())


def _norm_grad(d, x, weight, offset):
    """Gradients of x * rms(x) * (offset + weight) from d: of x, and of weight."""
    xh = x * _rms(x)
    g = _scaled(d, weight, offset)
    dx = _rms(x) * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    return dx, None if weight is None else (d * xh).sum(dim=0)


def _present(*outs):
    """The outputs that the case has."""
    return tuple(o for o in outs if o is not None)


def _norm(st):
    c = st["case"]
    x = st["x"].float()
    if c["way"] == "fwd":
        return _scaled(x * _rms(x), st["weight"], c["offset"]).to(torch.bfloat16)
    dx, dw = _norm_grad(st["dy"].float(), x, st["weight"], c["offset"])
    return _present((st["dres"].float() + dx).to(st["x"].dtype), dw)


def _block(st):
    c = st["case"]
    T, emb = c["T"], c["emb"]
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    if c["way"] == "fwd":
        if c["k"]:
            y = torch.zeros((T, emb), dtype=torch.float32, device=DEV)
            rows = st["slot_row"].long().view(T, c["k"])
            for j in range(c["k"]):
                y += st["topk_w"][:, j:j + 1] * st["ys"][rows[:, j]].float()
        else:
            y = st["y"].float()
        z = _scaled(y * _rms(y), st["post_weight"], c["offset"]) if c["post"] else y
        out = c["res_scale"] * st["res"].float() + c["scale"] * gate * z
        xn = _scaled(out * _rms(out), st["next_weight"], c["offset"]).to(torch.bfloat16) if c["next"] else None
        return _present(out.to(st["res"].dtype), xn)
    d = st["dout"].float()
    dnw = None
    if c["next"]:
        dx, dnw = _norm_grad(st["dnext"].float(), st["res"].float(), st["next_weight"], c["offset"])
        d = d + dx
    y = st["y"].float()
    dz = c["scale"] * gate * d
    z, dy, dpw = y, dz, None
    if c["post"]:
        z = _scaled(y * _rms(y), st["post_weight"], c["offset"])
        dy, dpw = _norm_grad(dz, y, st["post_weight"], c["offset"])
    dgate = None
    if c["gate"] != "none":
        dgate = c["scale"] * d * z
        if c["gate"] == "full":
            dgate = dgate.to(st["gate"].dtype)
        else:
            dgate = dgate.sum(dim=0) if c["gate"] == "channel" else dgate.sum(dim=1, keepdim=True)
    return _present((c["res_scale"] * d).to(st["res"].dtype), dy.to(torch.bfloat16), dpw, dgate, dnw)


# ------------------------------------------------------------------ the framework's calls

def _own(st):
    import mixture_experts_ffn_group_amd as moe
    c = st["case"]
    if c["op"] in ("few", "few_mx"):
        route = dict(topk_idx=st["idx"], topk_w=st["w"]) if c["routed"] else \
            dict(k=c["k"], wr=st["wr"], bias=st["bias"])
        if c["op"] == "few":
            r = moe.ffn_fwd_few(st["x"], st["wi"], st["wo"], **route)
        else:
            r = moe.ffn_fwd_few_mx(st["x"], st["wq"], **route)
        return r[0] if c["routed"] else r
    if c["op"] == "norm":
        if c["way"] == "fwd":
            return moe.norm(st["x"], st["weight"], offset=c["offset"], eps=EPS)
        return _present(*moe.norm_bwd(st["dy"], st["x"], st["weight"], offset=c["offset"], eps=EPS, dres=st["dres"]))
    how = dict(post_norm=c["post"], post_weight=st["post_weight"], gate=st["gate"], scale=c["scale"],
               res_scale=c["res_scale"], next_norm=c["next"], next_weight=st["next_weight"], offset=c["offset"], eps=EPS)
    if c["way"] == "fwd":
        if c["k"]:
            how.update(ys=st["ys"], slot_row=st["slot_row"], topk_w=st["topk_w"])
        r = moe.block_out(st["res"], st["y"], **how)
        return _present(r["out"], r["xn"])
    g = moe.block_out_bwd(st["dout"], st["y"], out=st["res"] if c["next"] else None, dxn=st["dnext"], **how)
    return _present(g["dres"], g["dy"], g["dpost_weight"], g["dgate"], g["dnext_weight"])


_PLAIN = {"few": _few, "few_mx": _few, "norm": _norm, "block": _block}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_picks(c, st):
    l = torch.stack([torch.mv(st["wr"].double().t(), row) for row in st["x"].double()])
    if st["bias"] is not None:
        l = l + st["bias"].double()[None, :]
    ids = torch.arange(c["E"], device=DEV)
    left, picks = l.clone(), []
    for _ in range(c["k"]):
        p = torch.where(left == left.amax(dim=1, keepdim=True), ids, c["E"]).amin(dim=1)
        left.scatter_(1, p[:, None], -math.inf)
        picks.append(p)
    idx = torch.stack(picks, dim=1)
    return idx.to(torch.int32), torch.softmax(l.gather(1, idx), dim=1)


def _e4m3_table():
    v = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-mag if code >> 7 else mag)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_mx(codes, scales, table):
    """[K, N] of one expert."""
    sc = torch.exp2(scales[..., :2].double() - 127)               # [K/64, N, 2]
    sc = sc.permute(0, 2, 1).reshape(-1, sc.shape[1])             # [K/32, N]
    return table[codes.long()].t() * sc.repeat_interleave(MX_BLOCK, dim=0)


def _exact_few(c, st):
    idx, w = (st["idx"], st["w"].double()) if c["routed"] else _exact_picks(c, st)
    table = _e4m3_table()
    y = torch.zeros((c["T"], c["emb"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        if c["op"] == "few":
            wi, wo = st["wi"][e].double(), st["wo"][e].double()
        else:
            q = st["wq"]
            wi = _exact_mx(q["wi_codes"][e], q["wi_scales"][e], table)
            wo = _exact_mx(q["wo_codes"][e], q["wo_scales"][e], table)
        g, u = torch.mm(st["x"][t].double(), wi).split(c["mlp"], dim=1)
        y.index_add_(0, t, w[t, j][:, None] * torch.mm(g / (1 + torch.exp(-g)) * u, wo))
    return y if c["routed"] else (y, idx, w)


def _autograd(fn, inputs, grads):
    """fn's gradients with respect to the tensors among inputs, by differentiation."""
    leaves = [None if v is None else v.detach().double().requires_grad_(True) for v in inputs]
    outs = fn(*leaves)
    total = sum((o * g.double()).sum() for o, g in zip(outs, grads) if g is not None)
    got = torch.autograd.grad(total, [v for v in leaves if v is not None], allow_unused=True)
    it = iter(got)
    return [None if v is None else next(it) for v in leaves]


def _exact_rms(v, weight, offset):
    n = v / ((v ** 2).sum(dim=-1, keepdim=True) / v.shape[-1] + EPS).sqrt()
    return n if weight is None else n * (weight + offset)


def _chunks(T, emb):
    """Row ranges of about 2^24 elements: what 64-bit differentiation holds at once stays small."""
    step = max(1, (1 << 24) // emb)
    return [slice(i, min(i + step, T)) for i in range(0, T, step)]


def _exact_norm(c, st):
    wt = None if st["weight"] is None else st["weight"].double()
    if c["way"] == "fwd":
        return _exact_rms(st["x"].double(), wt, c["offset"])
    dx, dw = torch.empty_like(st["x"], dtype=torch.float64), None
    for r in _chunks(c["T"], c["emb"]):
        gx, gw = _autograd(lambda x, w: (_exact_rms(x, w, c["offset"]),), (st["x"][r], st["weight"]), (st["dy"][r],))
        dx[r] = st["dres"][r].double() + gx
        dw = gw if dw is None or gw is None else dw + gw
    return _present(dx, dw)


def _exact_block(c, st):
    off = c["offset"]

    def after(y, gate, pw):
        z = _exact_rms(y, pw, off) if c["post"] else y
        return c["scale"] * z if gate is None else c["scale"] * z * gate

    def dbl(v):
        return None if v is None else v.double()

    def part(v, r):
        return v if v is None or c["gate"] == "channel" else v[r]

    T, emb, k = c["T"], c["emb"], c["k"]
    sum_, xn = torch.empty((T, emb), dtype=torch.float64, device=DEV), None
    if c["way"] == "fwd":
        xn = torch.empty_like(sum_) if c["next"] else None
        for r in _chunks(T, emb):
            if k:
                rows = st["slot_row"].view(T, k)[r].long()
                y = torch.matmul(st["topk_w"][r].double()[:, None, :], st["ys"][rows].double())[:, 0]
            else:
                y = st["y"][r].double()
            sum_[r] = c["res_scale"] * st["res"][r].double() + after(y, part(dbl(st["gate"]), r), dbl(st["post_weight"]))
            if c["next"]:
                xn[r] = _exact_rms(sum_[r], dbl(st["next_weight"]), off)
        return _present(sum_, xn)
    dy = torch.empty_like(sum_)
    dpw = dnw = dgate = None
    pieces = []
    for r in _chunks(T, emb):
        d = st["dout"][r].double()
        if c["next"]:
            gx, gw = _autograd(lambda x, w: (_exact_rms(x, w, off),), (st["res"][r], st["next_weight"]),
                               (st["dnext"][r],))
            d = d + gx
            dnw = gw if dnw is None or gw is None else dnw + gw
        sum_[r] = c["res_scale"] * d
        dy[r], gg, gp = _autograd(lambda y, gate, pw: (after(y, gate, pw),),
                                  (st["y"][r], part(st["gate"], r), st["post_weight"]), (d,))
        dpw = gp if dpw is None or gp is None else dpw + gp
        pieces.append(gg)
    if c["gate"] == "channel":
        dgate = sum(pieces)
    elif c["gate"] != "none":
        dgate = torch.cat(pieces)
    return _present(sum_, dy, dpw, dgate, dnw)


_EXACT = {"few": _exact_few, "few_mx": _exact_few, "norm": _exact_norm, "block": _exact_block}


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))
