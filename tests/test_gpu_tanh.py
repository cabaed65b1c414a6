"""Capped scores where one row's lie far beyond the reach of the polynomial of tanh: the other rows
of its warp keep errors that do not grow with the cap."""
import math

import pytest
import torch

import cache4_reference as ref4
import score_reference as ref
from io_aware_attention_flashattention_b200 import api
from test_gpu_cache4 import dev, filled
from test_gpu_score import make, run

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def score_error(products, t, d, bias=0.0):
    """How far a capped score is off, whatever the cap: d products summed in 32 bits, 2^-23 of
    what is summed each; tanh is off by 1.05e-6 of itself (the polynomial by 1e-6, 8.4 * 2^-23,
    and its evaluation and the factors of cap and log2 e by 4 * 2^-23; above 0.8 the form on the
    exponential by 6.3e-7, which is 9.5e-7 = 8 * 2^-23 of tanh 0.8): 13 * 2^-23 of t; and 8 *
    2^-23 of the bias and for the exponential and its argument."""
    return 2.0 ** -23 * (d * products + 13 * t.abs() + 8 * (bias + 1))


@pytest.mark.parametrize("cap", [1e2, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("dtype,causal,H,Hkv,slopes", [(BF, True, 2, 1, False), (HF, False, 2, 2, False),
                                                       (HF, True, 2, 1, True)])
def test_ordinary_rows_beside_a_far_one(cap, dtype, causal, H, Hkv, slopes):
    """Row 70's scores pass the polynomial's reach, so every warp that holds it takes the other
    form. O and LSE, dQ, dK and dV within the bounds of the roundings (score_reference.gradients,
    with the scores' error as above in place of one that grows with the cap)."""
    N, d, scale = 190, 64, 0.125
    q, k, v, do = make(1, H, Hkv, N, d, dtype, seed=int(cap))
    of = torch.arange(H, device="cuda") // (H // Hkv)
    # along key 3: scores of about 8 times the factor, and those of the other keys far too
    q[0, :, 70] = (k[0, of, 3].float() * min(cap / 5, 1e4)).to(dtype)
    slope = torch.tensor([0.25, 0.0625], device="cuda") if slopes else torch.zeros(2, device="cuda")
    got = run(q, k, v, do, scale, causal, None, dict(softcap=cap, slopes=slope if slopes else None))
    mask = ref.visible(1, N, causal).cuda()
    values, _ = ref.gradients(q, k, v, do, mask, scale, cap, slope)
    o, lse, dq, dk, dv = values
    u, tiny = ref.unit(dtype)
    Q, K, V, G = q.double(), k.double(), v.double(), do.double()
    dot = lambda a, b: torch.einsum("bhid,bhjd->bhij", a, b)  # noqa: E731
    x = dot(Q, K[:, of]) * scale
    ordinary = torch.cat([x[0, :, :70], x[0, :, 71:]], 1)
    assert float(x[0, :, 70].abs().max()) > 0.06 * cap and float(ordinary.abs().max()) < 12
    th = torch.tanh(x / cap)
    at = torch.arange(N, device="cuda", dtype=torch.float64)
    bias = slope.double()[None, :, None, None] * (at[:, None] - at[None]).abs()
    t = cap * th - bias
    zero = torch.zeros_like(t)
    seen = mask[:, None].expand_as(t)
    err = torch.where(seen, score_error(dot(Q.abs(), K[:, of].abs()) * scale, cap * th, d, bias), zero)
    top = err.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(torch.where(seen, t - lse[..., None], zero)), zero)
    dp = dot(G, V[:, of])
    ds = p * (dp - (G * o).sum(-1, keepdim=True)) * (1 - th * th) * scale
    b_lse = 1.05 * top.squeeze(-1) + N * 2.0 ** -24 + 2.0 ** -22 * (lse.abs() + 1)
    e_p = u + 2 * top
    err_p = e_p * p + tiny * seen
    b_o = torch.einsum("bhij,bhjd->bhid", err_p + u * p, V[:, of].abs()) + u * o.abs() + tiny
    b_d = (G.abs() * b_o).sum(-1, keepdim=True) + d * 2.0 ** -23 * dot(G.abs(), V[:, of].abs()).amax(-1, keepdim=True)
    err_s = (p * b_d * scale + (e_p + u) * ds.abs() + tiny * seen * scale
             + p * (dp - (G * o).sum(-1, keepdim=True)).abs() * scale * 1.5e-6)
    share = (1, Hkv, H // Hkv, N, d)
    turn = lambda a, b: torch.einsum("bhij,bhid->bhjd", a, b).reshape(share).sum(2)  # noqa: E731
    bounds = [1.05 * b_o, b_lse,
              1.05 * torch.einsum("bhij,bhjd->bhid", err_s, K[:, of].abs()) + u * dq.abs() + tiny,
              1.05 * turn(err_s, Q.abs()) + u * dk.abs() + tiny, 1.05 * turn(err_p, G.abs()) + u * dv.abs() + tiny]
    for name, a, w, b in zip(("O", "LSE", "dQ", "dK", "dV"), got, values, bounds):
        over = (a.double() - w).abs() - b
        assert torch.isfinite(a).all() and over.max() <= 0, f"{name}: {float(over.max()):.3g} over its bound"


@pytest.mark.parametrize("cap", [1e2, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_cache_heads_beside_a_far_one(cap, dtype):
    """Over the 4-bit cache: one head of eight that share a K/V head has far scores."""
    H, d, page, L = 8, 64, 16, 300
    codes, params, order, g = filled(20, 1, page, d, dtype, seed=3)
    params[..., 1] = (params[..., 0].float() * -7.5).to(dtype)
    q = torch.randn(1, H, 1, d, generator=g, device="cuda").to(dtype)
    q[0, 3] = (q[0, 3].float() * min(cap / 20, 1e4)).to(dtype)
    table = order.reshape(1, 20).contiguous()
    o, lse = api.cache4_attend(q, codes, params, table, dev([L]), scale=0.125, softcap=cap)
    assert api.fa_get_status() == 0
    c, s, z = ref4.rows(codes, params, table[0], L)
    for h in range(H):
        x = q[0, h, 0].double()
        t = cap * torch.tanh((s[0, 0] * c[0, 0] + z[0, 0]) @ x * 0.125 / cap)
        # summed: products q (code - 8) times the scale, and sum q times zero + 8 scale
        size = x.abs().sum() * (16 * s[0, 0] + z[0, 0].abs()).squeeze(-1) * 0.125
        err = float(score_error(size * (d + 8) / d, t, d).max())
        want = torch.logsumexp(t, 0)
        assert abs(float(lse[0, h, 0]) - float(want)) <= 1.05 * err + (L + 8) * 2.0 ** -23 + 2.0 ** -22 * abs(float(want)), h
