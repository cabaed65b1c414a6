"""Rows of the 4-bit cache whose range passes the largest 32-bit float."""
import pytest
import torch

from io_aware_attention_flashattention_b200 import api

pytestmark = pytest.mark.gpu


def quantise(x):
    """(code, scale, zero) of bf16 rows whose range may pass 32 bits: the definition's steps with
    x and scale halved, which changes no quotient (halving is exact at this size)."""
    f = x.float()
    low, high = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    fifteenth = torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)
    scale = (high * fifteenth - low * fifteenth).to(x.dtype)
    code = torch.round((0.5 * f - 0.5 * low) / (0.5 * scale.float())).clamp(0, 15)
    return code, scale, low


@pytest.mark.parametrize("d", [64, 128])
def test_rows_whose_range_passes_32_bits(d):
    top = torch.finfo(torch.bfloat16).max
    g = torch.Generator(device="cuda").manual_seed(d)
    k = torch.zeros(1, 1, 40, d, dtype=torch.float64, device="cuda")
    k[0, 0, 0, :3] = torch.tensor([3e38, -3e38, 1e38])
    k[0, 0, 1, :16] = torch.arange(16, device="cuda", dtype=k.dtype) * (2 * top / 15) - top  # every code
    k[0, 0, 2, :31] = (torch.arange(31, device="cuda", dtype=k.dtype) / 15 - 1) * top
    k[0, 0, 3:] = (torch.rand(37, d, generator=g, device="cuda", dtype=torch.float64) * 2 - 1) * top
    k[0, 0, 3:, 0], k[0, 0, 3:, 1] = top, -top
    k[0, 0, 20:, 1] = -top / 64  # ranges between the largest number and one and a bit of it
    k = k.clamp(-top, top).to(torch.bfloat16)
    codes, params = api.cache4_empty(1, 1, 64, d)
    table, pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    api.cache4_append(codes, params, k, k, table, pos)
    assert api.fa_get_status() == 0
    want, scale, zero = quantise(k[0, 0])
    got = torch.stack([codes[0, 0, 0, :40] & 15, codes[0, 0, 0, :40] >> 4], -1).flatten(-2)
    assert torch.equal(got.float(), want)
    # and against 64 bits: the quotient's own rounding is 15 * 2^-23 at most
    exact = (k[0, 0].double() - zero.double()) / scale.double()
    assert ((got.double() - exact).abs()[exact <= 15] <= 0.5 + 15 * 2.0 ** -23).all()
    assert got[0, :3].tolist() == [15, 0, 10] and sorted(set(got[1, :16].tolist())) == list(range(16))
    back = api.cache4_read(codes, params, table, pos, 40)[0][0, 0]
    value = (2 * (want * (0.5 * scale.float()) + 0.5 * zero.float())).to(torch.bfloat16)
    assert torch.equal(back, value)
