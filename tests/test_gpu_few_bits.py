"""How many bits the few-token layer keeps between its two products, by sums that are exact in fp32 in any order."""
import numpy as np
import pytest
import torch

import few_util as fu
import mixture_experts_ffn_group_amd as moe
import oracle
from test_gpu_few import _mx_values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# slices of 64 and of 128 columns, tiles of 16 and of 32 rows, both products in one kernel and in two
@pytest.mark.parametrize("T,emb,mlp", [(16, 64, 64), (9, 1088, 192), (1, 4096, 128), (16, 64, 19264), (48, 192, 128),
                                       (48, 1024, 64), (48, 192, 19200)])
@pytest.mark.parametrize("mx", [False, True])
def test_swiglu_output_enters_the_down_product_in_24_bits(T, emb, mlp, mx):
    """Two columns of the SwiGLU output, a0 = g u0 and a1 = g u1, with u0 - u1 = 2^-15: y = a0 - a1 = g 2^-15.

    silu(g) = g from g = 64 on (e^-64 is below half a step of 1). g has 4 bits and u 17, so a has at most 21; every partial
    sum of both products is a multiple of its last bit and fits 24 bits. 16 bits of a would leave y off by up to an
    eighth of itself."""
    gen = torch.Generator().manual_seed(T + emb)
    r = lambda *s: torch.randint(0, 8, s, generator=gen).float() / 8  # noqa: E731
    x = torch.zeros((T, emb))
    wi, wo = torch.zeros((1, emb, 2 * mlp)), torch.zeros((1, mlp, emb))
    g = 64 * (1 + r(T))
    cols = (0, mlp - 1)
    for t in range(T):  # four rows of wi a token: u = c0 + 2^-4 c1 + 2^-8 c2 + 2^-12 c3
        x[t, 4 * t:4 * t + 4] = 2.0 ** (-4 * torch.arange(4))
        u = 1 + r(4)
        u[3] = 1 + torch.randint(1, 8, (), generator=gen).float() / 8
        for i, c in enumerate(cols):
            wi[0, 4 * t, c] = g[t]
            wi[0, 4 * t:4 * t + 4, mlp + c] = u - torch.tensor([0, 0, 0, i / 8])
    wo[0, cols[0]], wo[0, cols[1]] = 1, -1
    x, wi, wo = (v.to(torch.bfloat16).to(DEV) for v in (x, wi, wo))
    idx, w = torch.zeros((T, 1), dtype=torch.int32, device=DEV), torch.ones((T, 1), device=DEV)
    if mx:
        # MXFP8 holds 3 bits behind the leading one, but of a block's largest power of two only up to 1.75: 1.875 saturates
        wq = moe.mx_quantize_expert_weights(wi, wo)
        y = moe.ffn_fwd_few_mx(x, wq, topk_idx=idx, topk_w=w)[0]
        wi, wo = _mx_values(wq, "wi"), _mx_values(wq, "wo")
    else:
        y = moe.ffn_fwd_few(x, wi, wo, topk_idx=idx, topk_w=w)[0]
        wi, wo = fu.f64(wi), fu.f64(wo)
    h = fu.f64(x) @ wi[0]
    ref = (h[:, :mlp] * h[:, mlp:]) @ wo[0]  # exact in 64 bits
    assert np.array_equal(ref, ref.astype(np.float32)) and (ref != 0).any()
    assert np.array_equal(fu.f64(y), ref)


@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (8, 200, 8), (20, 256, 13), (64, 70, 64)])
@pytest.mark.parametrize("bias", [False, True])
def test_logits_are_compared_in_all_64_bits(T, E, k, bias):
    """Logits +-1 + d 2^-50, d = 0..7, are exact in 64 bits: the larger d is picked first, equal ones by id."""
    gen = torch.Generator().manual_seed(T)
    emb, mlp = 64, 64
    x, wr = torch.zeros((T, emb)), torch.zeros((emb, E))
    x[:, 0] = torch.randint(0, 2, (T,), generator=gen).float() * 2 - 1
    x[:, 1] = 1
    d = torch.randint(0, 8, (E,), generator=gen).float() * 2.0 ** -50
    wr[0], b = 1, None
    if bias:
        b = d
    else:
        wr[1] = d
    ri, _ = fu.route(fu.f64(x), fu.f64(wr), fu.f64(b), k)
    wi, wo = torch.zeros((E, emb, 2 * mlp)).bfloat16().to(DEV), torch.zeros((E, mlp, emb)).bfloat16().to(DEV)
    y, idx, w = moe.ffn_fwd_few(x.bfloat16().to(DEV), wi, wo, k, wr=wr.to(DEV), bias=None if b is None else b.to(DEV))
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.abs(fu.f64(w) - 1 / k).max() <= 2 * fu.U / k and not y.any()


@pytest.mark.parametrize("code", [0, 1, 2, 3, 7, 12, 127, 246])
def test_mx_weights_of_every_scale(code):
    """All positive codes on one scale, one to a column: exact, but rounded to multiples of 2^-133 (half a step off at
    most) where the scale is below 2^-124. y = 64 x w, x a power of two: nothing else is rounded."""
    emb = mlp = 128
    wi = torch.zeros((1, emb, 2 * mlp))
    wi[0, 32, :mlp] = 64  # the gate, in a block of its own: silu(64) = 64
    wq = moe.mx_quantize_expert_weights(wi.bfloat16().to(DEV), torch.eye(emb)[None].bfloat16().to(DEV))
    wq["wi_codes"][0, mlp:, 0] = (torch.arange(mlp) % 127).to(torch.uint8).to(DEV)  # 127 is a NaN
    wq["wi_scales"][0, 0, mlp:, 0] = code
    x = torch.zeros((1, emb))
    x[0, 0], x[0, 32] = 2.0 ** (100 if code < 64 else -100), 1
    idx, w = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV)
    y = fu.f64(moe.ffn_fwd_few_mx(x.bfloat16().to(DEV), wq, topk_idx=idx, topk_w=w)[0])[0]
    v = np.array([oracle.e4m3_value(c % 127) for c in range(mlp)]) * 2.0 ** (code - 127)
    got = y / (64 * float(x[0, 0]))
    if code < 3:
        assert np.abs(got - v).max() == 2.0 ** -134 and np.array_equal(got, np.round(v * 2.0 ** 133) * 2.0 ** -133)
    else:
        assert np.array_equal(got, v) and got[126] > 0
