"""The weights of the attention over the 4-bit cache enter their product as two bf16 parts: the
output within a bound that one part would not keep."""
import math

import pytest
import torch

import cache4_reference as ref4
from io_aware_attention_flashattention_b200 import api

BF, HF = torch.bfloat16, torch.float16


# queries of a sixteenth: the bound on the scores' error stays below what one part loses


def rows_of(n_pages, Hkv, page, d, dtype, seed, device):
    """A cache of values about 0 (zero near -7.5 scale), so that outputs and their rounding are
    small next to the weights' products with code - 8."""
    g = torch.Generator().manual_seed(seed)
    codes, params = api.cache4_empty(n_pages, Hkv, page, d, dtype, device="cpu")
    codes.random_(0, 256, generator=g)
    scale = torch.rand(params.shape[:-1], generator=g) * 0.3 + 0.05
    params[..., 0] = scale.to(dtype)
    params[..., 1] = (-7.5 * scale + 0.02 * torch.randn(scale.shape, generator=g)).to(dtype)
    return codes.to(device), params.to(device), g


def head(q, c, s, z, scale, h, group):
    """(weights, K/V rows in 64 bits, bound on a score's error) of one query over all keys."""
    hk = h // group
    t = ((s[0, hk] * c[0, hk] + z[0, hk]) @ q.double()) * scale
    # a score: d products q (code - 8) in 32 bits, times the scale, plus sum q times zero + 8
    # scale (d + 8 roundings of what is summed); and 8 for the exponential and its argument
    size = q.double().abs().sum() * (16 * s[0, hk] + z[0, hk].abs()).squeeze(-1) * scale
    err = 2.0 ** -23 * ((q.numel() + 8) * size + 8 * (t.abs() + 1)).max()
    return torch.softmax(t, 0), c[1, hk], s[1, hk], z[1, hk], err


def bound(p, c, s, z, err, o, dtype):
    """The parts of a weight times its value's scale lose 2^-17 of it: the first is off by at most
    2^-8 of its power of two, 2^e, and the second holds that to 2^(e - 17). The rest is in 32 bits: the
    weights (twice a score's error: their own and their sum's), sums over L tokens; then the
    output's rounding."""
    u, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    L = p.numel()
    part = p @ (s * (c - 8).abs())
    every = p @ (s * (c - 8).abs() + 8 * s + z.abs())
    return 1.05 * (2.0 ** -17 * part + (2 * err + (L + 8) * 2.0 ** -23) * every) + u * o.abs() + tiny


def modelled(p, c, s, z, dtype, parts):
    """The output with the weights times the scales in `parts` bf16 numbers; the rest in 64 bits."""
    w = p[:, None] * s
    first = w.to(BF).double()
    used = first if parts == 1 else first + (w - first).to(BF).double()
    return ((used * (c - 8)).sum(0) + (p[:, None] * (z + 8 * s)).sum(0)).to(dtype).double()


LENGTHS = [1, 2, 5, 40, 333]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("L", LENGTHS)
def test_the_bound_tells_one_part_from_two(dtype, L):
    """A model of the arithmetic in which the second part is left out breaks the bound in f16
    (bf16's own rounding covers it, and over long rows the errors of many weights even out);
    with both parts it holds."""
    page, d = 16, 64
    codes, params, g = rows_of(-(-L // page), 2, page, d, dtype, L, "cpu")
    c, s, z = ref4.rows(codes, params, torch.arange(codes.shape[0]), L)
    over = {1: 0, 2: 0}
    for h in range(8):
        q = (torch.randn(d, generator=g) / 16).to(dtype)
        p, vc, vs, vz, err = head(q, c, s, z, d ** -0.5, h, 4)
        o = p @ (vs * vc + vz)
        b = bound(p, vc, vs, vz, err, o, dtype)
        for parts in over:
            over[parts] += int(((modelled(p, vc, vs, vz, dtype, parts) - o).abs() > b).sum())
    assert over[2] == 0
    assert dtype == BF or L > 40 or over[1] > 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [2, 16, 24])
def test_outputs_keep_the_bound(dtype, d, H):
    page, Hkv = 16, 2 if H < 24 else 1
    per = -(-max(LENGTHS) // page)
    codes, params, g = rows_of(per * len(LENGTHS), Hkv, page, d, dtype, H + d, "cuda")
    table = torch.arange(per * len(LENGTHS), dtype=torch.int32, device="cuda").reshape(len(LENGTHS), per)
    q = (torch.randn(len(LENGTHS), H, 1, d, generator=g) / 16).to(dtype).cuda()
    lengths = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    o, _ = api.cache4_attend(q, codes, params, table, lengths)
    assert api.fa_get_status() == 0
    for b, L in enumerate(LENGTHS):
        c, s, z = ref4.rows(codes, params, table[b], L)
        for h in range(H):
            p, vc, vs, vz, err = head(q[b, h, 0], c, s, z, 1 / math.sqrt(d), h, H // Hkv)
            want = p @ (vs * vc + vz)
            over = (o[b, h, 0].double() - want).abs() - bound(p, vc, vs, vz, err, want, dtype)
            assert over.max() <= 0, (L, h, float(over.max()))
