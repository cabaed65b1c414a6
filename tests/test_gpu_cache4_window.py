"""Attention over the 4-bit cache with a window: pages wholly in front of every row's window are
not looked at, whatever their table entries hold."""
import math

import pytest
import torch

from io_aware_attention_flashattention_b200 import api
from test_gpu_cache4 import BF, HF, check_attend, dev, filled

pytestmark = pytest.mark.gpu

WILD = [-1, 2**31 - 1, -2**31, 10**6]


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("Nq,left", [(1, 10), (1, 0), (3, 20), (5, 33)])
def test_entries_in_front_of_the_window_hold_anything(d, dtype, page, Nq, left):
    """The first token that a row sees moves over two steps of 32 tokens; every page in front of
    it has gone. The result is that of a whole table, and no bad page is noted."""
    B, H, Hkv, per = 2, 4, 2, 12
    codes, params, order, g = filled(B * per, Hkv, page, d, dtype, seed=left)
    whole = order.reshape(B, per).contiguous()
    q = torch.randn(B, H, Nq, d, generator=g, device="cuda").to(dtype)
    for n in range(90, 90 + 64, 5):
        lengths = [n, n + 16]
        table = whole.clone()
        for b, L in enumerate(lengths):
            first = max(0, L - Nq - left)
            for p in range(first // page):
                table[b, p] = WILD[p % 4]
            table[b, -(-L // page):] = WILD[b]
        o, lse = check_attend(q, codes, params, table, lengths, window_left=left)
        a, b = api.cache4_attend(q, codes, params, whole, dev(lengths), scale=1 / math.sqrt(d), window_left=left)
        assert torch.equal(o, a) and torch.equal(lse, b)
    assert api.fa_get_status() == 0


def test_a_page_that_the_window_reaches_is_still_noted():
    """The last token of a page that has gone is seen by the draft's first row alone."""
    codes, params, order, g = filled(8, 1, 16, 64, BF, seed=1)
    table = order.reshape(1, 8).clone()
    table[0, 4] = -1  # tokens 64 .. 79
    q = torch.randn(1, 2, 2, 64, generator=g, device="cuda").to(BF)
    check_attend(q, codes, params, table, [101], window_left=20, gone=[(0, 4)], status=5)  # from 79 on
    check_attend(q, codes, params, table, [101], window_left=19)                           # from 80 on
