"""8-bit activation checkpoints on the GPU against plain 64-bit implementations.

Codes, scales and values read back come from exact operations (a maximum, a power-of-two rescaling, one rounding)
and must be equal bit for bit. Tolerances of the rest: a bf16 output is off by half a step, 2^-8 of its value, plus
the fp32 arithmetic before it (stated at each check).
"""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_group_amd as moe
import scored_util as su

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _rows(M, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(rng.uniform(-30, 30, (M, 1)))
    special = [np.zeros(K), np.full(K, -0.0), np.where(np.arange(K) % 2, 3e38, -1e-30),
               np.full(K, 127.5 / 64), np.full(K, 1.9999999), 2.0 ** -126 * rng.standard_normal(K),
               2.0 ** -140 * rng.integers(-8, 9, K), (rng.integers(-254, 255, K)) / 128.0]  # ties of the rounding
    for i, s in enumerate(special[:M]):
        x[i] = s
    return torch.from_numpy(x.astype(np.float32))


@pytest.mark.parametrize("M,K", [(1, 32), (8, 64), (9, 96), (300, 1536), (129, 7168), (5, 2080), (1000, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_and_read_back(M, K, dtype):
    x = _rows(M, K, M + K).to(dtype)
    codes, scales = moe.ckpt_quantize(x.to(DEV))
    rc, rs = su.ckpt_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    ref = su.ckpt_values(rc, rs)
    for out in (torch.float32, torch.bfloat16):
        v = moe.ckpt_dequantize(codes, scales, dtype=out)
        assert v.dtype == out and np.array_equal(v.cpu().double().numpy(), ref)
    # half a step, or one past 127.5 steps
    err = np.abs(x.double().numpy() - ref).reshape(M, -1, 32)
    step = np.ldexp(1.0, rs.astype(np.int64) - 133)[:, :, None]
    sat = np.abs(x.double().numpy()).reshape(M, -1, 32) > 127.5 * step
    assert (err <= np.where(sat, 1.0, 0.5) * step).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_non_finite_blocks_read_back_as_nan(dtype):
    x = torch.randn((6, 128), generator=torch.Generator().manual_seed(0)).to(dtype)
    x[1, 40] = float("nan")
    x[2, 0] = float("inf")
    x[3, 127] = -float("inf")
    x[4] = torch.finfo(dtype).max
    codes, scales = moe.ckpt_quantize(x.to(DEV))
    rc, rs = su.ckpt_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)
    v = moe.ckpt_dequantize(codes, scales, dtype=torch.float32).cpu().double().numpy()
    assert np.array_equal(v, su.ckpt_values(rc, rs), equal_nan=True)
    assert np.isnan(v[1, 32:64]).all() and np.isfinite(v[1, :32]).all() and np.isfinite(v[4]).all()


def test_read_back_through_a_row_mapping():
    T, K, k = 50, 96, 3
    x = _rows(T, K, 2)
    codes, scales = moe.ckpt_quantize(x.to(DEV))
    slots = np.random.default_rng(1).permutation(T * k).astype(np.int32)
    slots[:3] = [-9, 10 ** 6, 2 ** 31 - 1]  # clamped into the checkpoint
    v = moe.ckpt_dequantize(codes, scales, torch.from_numpy(slots).to(DEV), k)
    rows = np.clip(np.trunc(slots / k).astype(np.int64), 0, T - 1)
    ref = su.ckpt_values(*su.ckpt_quantize(x.double().numpy()))[rows]
    assert np.array_equal(v.cpu().double().numpy(), ref)
    assert moe.ckpt_dequantize(codes, scales, torch.zeros(0, dtype=torch.int32, device=DEV)).shape == (0, K)


def test_no_rows():
    c, s = moe.ckpt_quantize(torch.zeros((0, 64), device=DEV))
    assert c.shape == (0, 64) and s.shape == (0, 2)
    assert moe.ckpt_dequantize(c, s).shape == (0, 64)
    dh, a, ds = moe.swiglu_bwd_ckpt(torch.zeros((0, 32), dtype=torch.bfloat16, device=DEV), c, s)
    assert dh.shape == (0, 64) and a.shape == (0, 32) and ds.shape == (0,)


def test_refused_shapes():
    x = torch.zeros((4, 64), device=DEV)
    c, s = moe.ckpt_quantize(x)
    with pytest.raises(moe.MoeError):
        moe.ckpt_quantize(torch.zeros((4, 48), device=DEV))
    with pytest.raises(ValueError):
        moe.ckpt_dequantize(c, s[:, :1].contiguous())
    with pytest.raises(ValueError):
        moe.ckpt_quantize(x.t())
    da = torch.zeros((4, 32), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        moe.swiglu_bwd_ckpt(da[:3], c, s)
    with pytest.raises(ValueError):
        moe.swiglu_bwd_ckpt(da, c, s, slot_scale=torch.ones(3, device=DEV))
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        moe.grouped_gemm_wgrad_ckpt(c, s, da, off, 3)
    with pytest.raises(moe.MoeError):
        moe.grouped_gemm_wgrad_ckpt(c, s, torch.cat([da, da]), off, 2)  # 8 rows, 4 in the checkpoint


# ------------------------------------------------------------------ SwiGLU backward

def _swiglu_case(M, mlp, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    h = torch.from_numpy((rng.standard_normal((M, 2 * mlp)) * spread).astype(np.float32))
    codes, scales = su.ckpt_quantize(h.double().numpy())
    da = torch.from_numpy(rng.standard_normal((M, mlp)).astype(np.float32)).to(torch.bfloat16)
    slot = rng.permutation(M).astype(np.int32)
    w = rng.uniform(0, 1, M).astype(np.float32)
    return codes, scales, da, slot, w


def _swiglu_ref(codes, scales, da, slot, w):
    M, mlp = da.shape
    h = su.ckpt_values(codes, scales)
    g, u = h[:, :mlp], h[:, mlp:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    d = da.double().numpy()
    q = np.arange(M) if slot is None else slot
    wr = np.ones(M) if w is None else w.astype(np.float64)[q]
    a = g * s * u
    dh = np.concatenate([wr[:, None] * d * u * s * (1 + g * (1 - s)), wr[:, None] * d * g * s], axis=1)
    # magnitudes of the terms the fp32 arithmetic adds up: 1 + g (1 - s) cancels near its zero
    mag = np.concatenate([np.abs(wr[:, None] * d * u * s) * (1 + np.abs(g) * (1 - s)), np.abs(dh[:, mlp:])], axis=1)
    ds = np.zeros(M)
    dm = np.zeros(M)
    ds[q] = (d * a).sum(axis=1)
    dm[q] = np.abs(d * a).sum(axis=1)
    # exp(-g) leaves fp32's range past g = -88, where the sigmoid, below 7e-39, may come out as 0
    flush = 7e-39 * (1 + np.abs(g)) * (1 + np.abs(u)) * (1 + np.abs(d))
    return dh, mag, a, ds, dm, flush


def _np_dev(v):
    return None if v is None else torch.from_numpy(v).to(DEV)


def _check_swiglu(codes, scales, da, slot, w):
    dh, a, ds = moe.swiglu_bwd_ckpt(da.to(DEV), _np_dev(codes), _np_dev(scales), _np_dev(slot), _np_dev(w))
    rdh, mag, ra, rds, dm, flush = _swiglu_ref(codes, scales, da, slot, w)
    # fp32 arithmetic: about ten roundings and an exponential, 2^-20 of the terms; then the bf16 rounding
    fp = 2.0 ** -20
    for got, ref, m, fl, name in ((dh, rdh, mag, np.concatenate([flush, flush], axis=1), "dh"),
                                  (a, ra, np.abs(ra), flush, "a")):
        err = np.abs(got.cpu().double().numpy() - ref)
        tol = 2.0 ** -8 * np.abs(ref) + 2 * fp * m + fl
        assert (err <= tol).all(), (name, (err / tol).max())
    mlp = da.shape[1]
    q = np.arange(da.shape[0]) if slot is None else slot
    fsum = np.zeros(da.shape[0])
    fsum[q] = flush.sum(axis=1)
    tol = (fp + mlp * 2.0 ** -24) * dm + fsum
    assert (np.abs(ds.cpu().double().numpy() - rds) <= tol).all()
    return dh, a, ds


@pytest.mark.parametrize("M,mlp", [(1, 32), (3, 64), (515, 256), (257, 768), (40, 2048), (100, 96), (7, 544)])
@pytest.mark.parametrize("mapped", [False, True])
def test_swiglu_bwd_ckpt(M, mlp, mapped):
    codes, scales, da, slot, w = _swiglu_case(M, mlp, M + mlp)
    _check_swiglu(codes, scales, da, slot if mapped else None, w if mapped else None)


def test_swiglu_bwd_ckpt_large_gates():
    """Saturated sigmoids of both signs: the results stay finite and right."""
    codes, scales, da, slot, w = _swiglu_case(64, 128, 3, spread=60.0)
    for v in _check_swiglu(codes, scales, da, slot, w):
        assert torch.isfinite(v.float()).all()


def test_swiglu_bwd_ckpt_zero_weight_rows_and_optional_outputs():
    codes, scales, da, slot, w = _swiglu_case(33, 96, 5)
    w[::3] = 0.0
    dh, a, ds = _check_swiglu(codes, scales, da, slot, w)
    assert (dh[torch.from_numpy(w[slot] == 0).to(DEV)] == 0).all()
    args = (da.to(DEV), _np_dev(codes), _np_dev(scales), _np_dev(slot), _np_dev(w))
    d2, none_a, none_s = moe.swiglu_bwd_ckpt(*args, want_a=False, want_dscale=False)
    assert none_a is None and none_s is None and torch.equal(d2, dh)


def test_swiglu_bwd_ckpt_nan_block_stays_visible():
    codes, scales, da, slot, w = _swiglu_case(4, 64, 6)
    codes[1, :32] = 0
    scales[1, 0] = 255  # the first gate block of row 1
    dh, a, ds = moe.swiglu_bwd_ckpt(da.to(DEV), _np_dev(codes), _np_dev(scales))
    assert torch.isnan(dh[1, :32].float()).all() and torch.isnan(a[1, :32].float()).all() and torch.isnan(ds[1])
    assert torch.isfinite(dh[1, 32:64].float()).all() and torch.isfinite(dh[2].float()).all()


def test_swiglu_bwd_ckpt_slots_out_of_range():
    codes, scales, da, slot, w = _swiglu_case(6, 64, 7)
    slot[:] = [0, -1, 2, 2 ** 31 - 1, 4, -2 ** 31]
    dh, a, ds = moe.swiglu_bwd_ckpt(da.to(DEV), _np_dev(codes), _np_dev(scales), _np_dev(slot), _np_dev(w))
    torch.cuda.synchronize()
    assert (dh[1::2] == 0).all()


def test_swiglu_bwd_ckpt_more_rows_than_one_launch_takes():
    """2^29 + 5 rows, past 2^32 lanes: the first and the last rows as in a call of their own."""
    M, mlp, n = 2 ** 29 + 5, 32, 300
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info(DEV)[0] < 180 << 30:
        pytest.skip("needs 140 GB of device memory")
    rng = torch.Generator().manual_seed(1)
    da = torch.zeros((M, mlp), dtype=torch.bfloat16, device=DEV)
    codes = torch.zeros((M, 2 * mlp), dtype=torch.int8, device=DEV)
    scales = torch.full((M, 2), 127, dtype=torch.uint8, device=DEV)
    for r in (slice(0, n), slice(M - n, M)):
        da[r] = torch.randn((n, mlp), generator=rng).to(torch.bfloat16)
        codes[r] = torch.randint(-127, 128, (n, 2 * mlp), generator=rng, dtype=torch.int8)
    dh, _, ds = moe.swiglu_bwd_ckpt(da, codes, scales, want_a=False)
    for r in (slice(0, n), slice(M - n, M)):
        small, _, dss = moe.swiglu_bwd_ckpt(*(t[r].clone() for t in (da, codes, scales)), want_a=False)
        assert torch.equal(dh[r], small) and torch.equal(ds[r], dss)
    del da, codes, scales, dh, ds
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ weight gradient

def _wgrad_case(T, k, E, P, Q, seed, sizes=None):
    rng = np.random.default_rng(seed)
    S = T * k
    x = torch.from_numpy(rng.standard_normal((T, P)).astype(np.float32))
    codes, scales = su.ckpt_quantize(x.double().numpy())
    slot = rng.permutation(S).astype(np.int32)
    if sizes is None:
        sizes = rng.multinomial(S, rng.dirichlet(np.ones(E)))
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    D = torch.from_numpy(rng.standard_normal((S, Q)).astype(np.float32)).to(torch.bfloat16)
    return codes, scales, slot, off, D


def _check_wgrad(codes, scales, slot, off, D, k, E, workspace=None):
    out = moe.grouped_gemm_wgrad_ckpt(_np_dev(codes), _np_dev(scales), D.to(DEV), _np_dev(off), E,
                                      row_slot=_np_dev(slot), slot_div=k, workspace=workspace)
    x = su.ckpt_values(codes, scales)
    xr = x if slot is None else x[slot // k]
    d = D.double().numpy()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        ref = xr[lo:hi].T @ d[lo:hi]
        mag = np.abs(xr[lo:hi]).T @ np.abs(d[lo:hi])
        got = out[e].cpu().double().numpy()
        # exact products, fp32 accumulation of hi - lo terms, one bf16 rounding
        tol = 2.0 ** -8 * np.abs(ref) + (hi - lo + 2) * 2.0 ** -24 * mag
        assert (np.abs(got - ref) <= tol).all(), (e, (np.abs(got - ref) / np.maximum(tol, 1e-300)).max())
        if hi == lo:
            assert (got == 0).all()
    return out


@pytest.mark.parametrize("T,k,E,P,Q", [(1, 1, 1, 32, 8), (40, 2, 3, 64, 64), (500, 3, 12, 256, 384),
                                       (300, 1, 5, 96, 40), (700, 4, 8, 544, 264), (64, 8, 61, 128, 136),
                                       (2000, 2, 2, 320, 512), (33, 2, 7, 800, 72)])
def test_wgrad_ckpt(T, k, E, P, Q):
    _check_wgrad(*_wgrad_case(T, k, E, P, Q, T + P), k, E)


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 161, 255])
def test_wgrad_ckpt_group_sizes(n):
    """Every number of rows around the k-slices, with an empty group on either side, and rows after the last group
    that must not enter."""
    k, E, P, Q = 2, 5, 288, 264
    rest = 64
    T = (n + 37 + 1 + rest + 1) // 2 + 1
    sizes = [0, n, 0, 37, 1]
    case = _wgrad_case(T, k, E, P, Q, n, sizes=sizes)
    _check_wgrad(*case, k, E)


def test_wgrad_ckpt_without_a_mapping():
    T, E, P, Q = 300, 4, 256, 128
    codes, scales, _, off, D = _wgrad_case(T, 1, E, P, Q, 3)
    _check_wgrad(codes, scales, None, off, D, 1, E)


def test_wgrad_ckpt_many_tiles_a_workgroup():
    """More output tiles than workgroups, of unlike k-lengths, so that workgroups go from tile to tile."""
    T, k, E, P, Q = 900, 2, 40, 1056, 1032
    _check_wgrad(*_wgrad_case(T, k, E, P, Q, 11), k, E)


@pytest.mark.parametrize("sizes,P,Q", [([3000, 500, 20, 0, 481], 256, 520), ([0, 0, 4096], 64, 64), ([4095], 160, 1032),
                                       ([1, 2, 2500, 1, 2500], 96, 8), ([900, 700, 800, 600, 1001], 288, 264)])
def test_wgrad_ckpt_long_groups_cut_along_their_rows(sizes, P, Q):
    """Groups longer than a workgroup's mean load, with every size of workspace: none, too small for the pieces
    wanted, and the one asked for (some of it past the end of what is needed); the same bits on every run."""
    E, M = len(sizes), sum(sizes)
    case = _wgrad_case(M, 1, E, P, Q, M, sizes=sizes)
    n = moe._lib.lib().moe_wgrad_ckpt_workspace_bytes(E, M, P, Q)
    assert n >= 1 << 18
    for bytes_ in (0, (1 << 18) + 16, 5 << 18, n, n + (1 << 20)):
        ws = torch.full((bytes_ + 4096,), 0x5a, dtype=torch.uint8, device=DEV)
        out = _check_wgrad(*case, 1, E, workspace=ws[:bytes_])
        assert (ws[bytes_:] == 0x5a).all()
        again = _check_wgrad(*case, 1, E, workspace=ws[:bytes_])
        assert torch.equal(out, again)


@pytest.mark.parametrize("E,M,P,Q,power", [(256, 6000, 32, 8, 1.5), (255, 9000, 64, 520, 1.1), (61, 12000, 96, 72, 2.0),
                                           (17, 20000, 160, 1032, 1.1), (64, 5000, 1056, 40, 0.0), (2, 9001, 288, 8, 3.0)])
def test_wgrad_ckpt_skewed_loads(E, M, P, Q, power):
    """Work lists of many and few experts in shuffled order of load, some cut, with the workspace asked for."""
    rng = np.random.default_rng(E + M)
    w = np.arange(1, E + 1) ** -power
    sizes = rng.permutation(rng.multinomial(M, w / w.sum()))
    case = _wgrad_case(M, 1, E, P, Q, M, sizes=sizes)
    n = moe._lib.lib().moe_wgrad_ckpt_workspace_bytes(E, M, P, Q)
    ws = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device=DEV)
    out = _check_wgrad(*case, 1, E, workspace=ws[:n])
    assert (ws[n:] == 0x5a).all()
    assert torch.equal(out, _check_wgrad(*case, 1, E, workspace=ws[:n]))


def test_wgrad_ckpt_rows_of_other_groups_never_enter():
    """NaN in a row of another group, in rows behind the last group and in a token no row reads."""
    k, E, P, Q = 1, 3, 64, 64
    codes, scales, _, off, D = _wgrad_case(200, k, E, P, Q, 5, sizes=[33, 50, 70])
    slot = np.arange(200, dtype=np.int32)
    scales[40, :] = 255        # group 1
    scales[160, :] = 255       # behind the last group
    D[170] = float("nan")
    out = moe.grouped_gemm_wgrad_ckpt(_np_dev(codes), _np_dev(scales), D.to(DEV), _np_dev(off), E,
                                      row_slot=_np_dev(slot), slot_div=1)
    assert torch.isfinite(out[0].float()).all() and torch.isfinite(out[2].float()).all()
    assert torch.isnan(out[1].float()).all()


def test_wgrad_ckpt_ends_of_the_scale_range():
    """Blocks at both ends of the scale codes (2^127 and more in magnitude; values that are subnormal), a code a
    group, with D scaled so that the sums stay in range; and codes of -128, which the quantizer never writes."""
    rng = np.random.default_rng(8)
    cs, n, P, Q = [254, 253, 247, 127, 8, 7, 2, 1], 40, 96, 72
    E, M = len(cs), len(cs) * n
    codes = rng.integers(-128, 128, (M, P)).astype(np.int8)
    codes[:n] = np.maximum(codes[:n], -127)  # -128 of the largest step is past bf16
    scales = np.repeat(np.array(cs, np.uint8), n)[:, None].repeat(P // 32, axis=1)
    d = rng.integers(1, 8, (M, Q)) * np.ldexp(1.0, np.minimum(137 - scales[:, :1].astype(np.int64), 120))
    D = torch.from_numpy(d).to(torch.bfloat16)
    off = (np.arange(E + 1) * n).astype(np.int32)
    _check_wgrad(codes, np.ascontiguousarray(scales), np.arange(M, dtype=np.int32), off, D, 1, E)


def test_wgrad_ckpt_no_rows():
    c, s = moe.ckpt_quantize(torch.zeros((0, 64), device=DEV))
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    D = torch.zeros((0, 40), dtype=torch.bfloat16, device=DEV)
    out = moe.grouped_gemm_wgrad_ckpt(c, s, D, off, 3)
    assert (out == 0).all()


def test_wgrad_ckpt_out_of_range_indices_stay_inside():
    codes, scales, slot, off, D = _wgrad_case(20, 2, 3, 64, 64, 4)
    slot[:4] = [-1, -2 ** 31, 2 ** 31 - 1, 10 ** 6]
    off[:] = [-5, 10, 8, 10 ** 6]  # clamped; a decreasing pair is an empty group
    out = moe.grouped_gemm_wgrad_ckpt(_np_dev(codes), _np_dev(scales), D.to(DEV), _np_dev(off), 3,
                                      row_slot=_np_dev(slot), slot_div=2)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all() and (out[1] == 0).all()


def test_graph_replays_and_streams_equal_eager():
    T, k, E, P, mlp = 200, 2, 6, 256, 128
    codes, scales, slot, off, _ = _wgrad_case(T, k, E, P, 2 * mlp, 4)
    hc, hs, da, _, w = _swiglu_case(T * k, mlp, 5)
    slot, off, hc, hs, w, da = (_np_dev(v) if isinstance(v, np.ndarray) else v.to(DEV)
                                for v in (slot, off, hc, hs, w, da))
    x = torch.randn((T, P), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)

    def step(xin):
        c, s = moe.ckpt_quantize(xin)
        dh, a, ds = moe.swiglu_bwd_ckpt(da, hc, hs, slot, w)
        return moe.grouped_gemm_wgrad_ckpt(c, s, dh, off, E, row_slot=slot, slot_div=k), dh, a, ds, \
            moe.ckpt_dequantize(c, s, slot, k)

    step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    for rep in range(4):
        xr = torch.randn((T, P), generator=torch.Generator().manual_seed(9 + rep)).to(torch.bfloat16).to(DEV)
        x.copy_(xr)
        graph.replay()
        torch.cuda.synchronize()
        ref = step(xr)
        for got, r in zip(out, ref):
            assert torch.equal(got, r), rep
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        o1 = step(x)
    with torch.cuda.stream(s2):
        o2 = step(x)
    torch.cuda.synchronize()
    for a, b, r in zip(o1, o2, step(x)):
        assert torch.equal(a, r) and torch.equal(b, r)


def test_cut_groups_in_a_graph_on_one_workspace():
    """A captured gradient whose groups are cut, replayed with other loads in between: some cut nothing, some other
    groups, all on the same workspace."""
    E, M, P, Q = 4, 5000, 128, 520
    codes, scales, slot, off, D = _wgrad_case(M, 1, E, P, Q, 3, sizes=[4000, 1000, 0, 0])
    codes, scales, slot, off, D = (_np_dev(v) if isinstance(v, np.ndarray) else v.to(DEV)
                                   for v in (codes, scales, slot, off, D))
    ws = torch.empty(moe._lib.lib().moe_wgrad_ckpt_workspace_bytes(E, M, P, Q), dtype=torch.uint8, device=DEV)

    def run(o, w):
        return moe.grouped_gemm_wgrad_ckpt(codes, scales, D, o, E, row_slot=slot, slot_div=1, workspace=w)

    run(off, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(off, ws)
    for sizes in ([0, 0, 5000, 0], [1250, 1250, 1250, 1250], [10, 20, 0, 4970], [0, 0, 0, 0], [4000, 1000, 0, 0]):
        o = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
        off.copy_(o)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run(o, None)), sizes


def test_outputs_end_where_they_should():
    """Every output inside a larger buffer, through the C interface: nothing past its end changes."""
    import ctypes as C
    lib = moe._lib.lib()
    st = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731

    def buf(n):
        return torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device=DEV)

    M, K = 37, 96
    x = _rows(M, K, 1).to(DEV)
    c, s, v = buf(M * K), buf(M * K // 32), buf(M * K * 2)
    assert lib.moe_ckpt_quantize(p(x), 0, M, K, p(c), p(s), st) == 0
    assert lib.moe_ckpt_dequantize(p(c), p(s), M, K, None, 1, M, p(v), 1, st) == 0
    mlp = K // 2 // 32 * 32
    da = torch.ones((M, mlp), dtype=torch.bfloat16, device=DEV)
    h = torch.zeros(M * 2 * mlp, dtype=torch.int8, device=DEV)
    hs = torch.full((M * mlp // 16,), 120, dtype=torch.uint8, device=DEV)
    dh, a, ds = buf(M * 2 * mlp * 2), buf(M * mlp * 2), buf(M * 4)
    assert lib.moe_swiglu_bwd_ckpt(M, mlp, p(da), p(h), p(hs), None, None, p(dh), p(a), p(ds), st) == 0
    E, Q = 3, 72
    off = torch.tensor([0, 20, 20, M], dtype=torch.int32, device=DEV)
    D = torch.ones((M, Q), dtype=torch.bfloat16, device=DEV)
    w = buf(E * K * Q * 2)
    assert lib.moe_grouped_gemm_wgrad_ckpt(p(c), p(s), M, None, 1, p(D), p(off), E, M, K, Q, p(w), None, 0, st) == 0
    torch.cuda.synchronize()
    for b in (c, s, v, dh, a, ds, w):
        assert (b[-4096:] == 0x5a).all()
