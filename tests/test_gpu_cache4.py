"""The 4-bit cache on the GPU: appended rows bit for bit as the definition quantises them,
nothing else written, and the attention over it within the bounds of its roundings
(cache4_reference.attend)."""
import math
import random

import pytest
import torch

import cache4_reference as ref4
import score_reference as ref
from io_aware_attention_flashattention_b200 import api

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
FA_ERR_BAD_PAGE = 5


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def filled(n_pages, Hkv, page, d, dtype, seed, spread=1.0):
    """A cache of random rows and codes, and a shuffled order of its pages."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes, params = api.cache4_empty(n_pages, Hkv, page, d, dtype)
    codes.random_(0, 256, generator=g)
    params[..., 0] = (torch.rand(params.shape[:-1], generator=g, device="cuda") * 0.3 * spread + 0.05).to(dtype)
    params[..., 1] = (torch.randn(params.shape[:-1], generator=g, device="cuda") - 2.5 * spread).to(dtype)
    return codes, params, torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32), g


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hkv,n,page,positions,counts", [
    (1, 1, 1, 16, [0], None),
    (3, 2, 1, 32, [31, 32, 95], None),
    (2, 3, 70, 64, [5, 60], [70, 33]),
    (4, 1, 40, 16, [0, 15, 16, 1], [0, 40, 1, -3]),
    (2, 2, 33, 256, [200, 223], [99, 12]),  # counts beyond n count as n
])
def test_append_and_read_bit_for_bit(dtype, d, B, Hkv, n, page, positions, counts):
    per = 6
    codes, params, order, g = filled(B * per + 2, Hkv, page, d, dtype, seed=n)
    table = order[:B * per].reshape(B, per).contiguous()
    k = (torch.randn(B, Hkv, n, d, generator=g, device="cuda") * 3 + 1).to(dtype)
    v = torch.randn(B, Hkv, n, d, generator=g, device="cuda").to(dtype)
    k[0, 0, 0], v[-1, -1, -1] = 0.0, -7.0  # rows without a spread
    want_c, want_p = codes.clone(), params.clone()
    for b in range(B):
        for t in range(n if counts is None else max(0, min(n, counts[b]))):
            at = positions[b] + t
            page_id, slot = int(table[b, at // page]), at % page
            for which, x in enumerate((k, v)):
                c, s, z = ref4.quantise(x[b, :, t])
                want_c[page_id, which, :, slot] = c[:, 0::2] | (c[:, 1::2] << 4)
                want_p[page_id, which, :, slot] = torch.cat([s, z], -1)
    pos, cnt = dev(positions), None if counts is None else dev(counts)
    api.cache4_append(codes, params, k, v, table, pos, counts=cnt)
    assert torch.equal(codes, want_c) and torch.equal(params, want_p)
    got = api.cache4_read(codes, params, table, pos, n, counts=cnt)
    for which, (x, back) in enumerate(zip((k, v), got)):
        c, s, z = ref4.quantise(x)
        value = (c.float() * s.float() + z.float()).to(dtype)
        for b in range(B):
            m = n if counts is None else max(0, min(n, counts[b]))
            assert torch.equal(back[b, :, :m], value[b, :, :m]) and (back[b, :, m:] == 0).all()
    assert api.fa_get_status() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_of_extreme_rows(dtype):
    """Rows over the type's whole range, tiny ones, and a NaN, which reads back as NaN."""
    top = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    k = torch.zeros(1, 1, 6, 64, dtype=dtype, device="cuda")
    k[0, 0, 0, ::2], k[0, 0, 0, 1::2] = top, -top
    k[0, 0, 1, 3] = tiny
    k[0, 0, 2] = torch.linspace(-1, 1, 64).to(dtype)
    k[0, 0, 3, 5] = float("nan")
    k[0, 0, 4] = top
    k[0, 0, 5, 63] = -1.0
    codes, params = api.cache4_empty(1, 1, 16, 64, dtype)
    table, pos = dev([[0]]), dev([0])
    api.cache4_append(codes, params, k, k, table, pos)
    got = api.cache4_read(codes, params, table, pos, 6)[0]
    c, s, z = ref4.quantise(k)
    value = (c.double() * s.double() + z.double()).to(dtype)  # 15 scales pass the range of 32 bits
    assert torch.equal(got[0, 0, [0, 1, 2, 4, 5]], value[0, 0, [0, 1, 2, 4, 5]])
    assert got[0, 0, 3].isnan().all()


def check_attend(q, codes, params, table, lengths, gone=(), status=0, max_len=None, **kw):
    scale = kw.pop("scale", 1.0 / math.sqrt(q.shape[-1]))
    o, lse = api.cache4_attend(q, codes, params, table, dev(lengths), scale=scale, max_len=max_len, **kw)
    torch.cuda.synchronize()
    assert api.fa_get_status() == status
    (want_o, want_l), (b_o, b_l) = ref4.attend(q, codes, params, table, lengths, scale, kw.get("window_left", -1),
                                               kw.get("softcap"), kw.get("slopes"), gone)
    empty = want_l == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (o[empty] == 0).all()
    over = (o.double() - want_o).abs() - b_o
    assert torch.isfinite(o).all() and over.max() <= 0, f"O {float(over.max()):.3g} over its bound"
    over = ((lse.double() - want_l).abs() - b_l)[~empty]
    assert over.numel() == 0 or over.max() <= 0, f"LSE {float(over.max()):.3g} over its bound"
    return o, lse


CASES = [
    # B, H, Hkv, Nq, d, type, page, lengths, the rest
    (1, 1, 1, 1, 64, BF, 16, [1], {}),
    (1, 8, 8, 1, 64, BF, 16, [127], {}),
    (2, 2, 2, 1, 128, HF, 16, [16, 17], {}),
    (3, 4, 1, 1, 128, BF, 32, [0, 31, 400], {}),
    (2, 8, 1, 1, 64, HF, 64, [65, 500], dict(softcap=30.0)),
    (1, 14, 2, 1, 128, BF, 64, [777], dict(softcap=5.0, slopes=True)),
    (2, 16, 1, 1, 128, BF, 128, [300, 129], dict(slopes=True)),
    (2, 17, 1, 1, 128, HF, 64, [70, 515], dict(softcap=8.0, slopes=True)),
    (1, 24, 1, 1, 64, BF, 16, [1500], {}),
    (3, 12, 2, 4, 64, HF, 32, [2, 33, 700], dict(window_left=64, slopes=True)),
    (2, 25, 1, 1, 128, BF, 64, [64, 321], dict(softcap=8.0)),
    (2, 64, 2, 1, 64, BF, 256, [513, 40], {}),
    (2, 4, 4, 5, 128, BF, 32, [3, 200], {}),  # a draft longer than its sequence
    (2, 6, 2, 8, 64, HF, 16, [8, 333], dict(window_left=100)),
    (1, 16, 4, 5, 128, BF, 32, [1030], dict(window_left=511)),
    (2, 4, 2, 1, 128, BF, 64, [64, 900], dict(window_left=0)),
    (2, 4, 2, 3, 128, BF, 64, [64, 900], dict(window_left=1000, softcap=10.0, slopes=True)),
    (1, 2, 1, 50, 64, BF, 16, [60], {}),
    (1, 2, 2, 3, 64, BF, 16, [100], dict(window_left=2**31 - 1)),
    (2, 2, 1, 40, 64, HF, 16, [30, 90], dict(window_left=2**31 - 2)),
    (1, 4, 1, 1, 128, HF, 128, [9000], dict(slopes=True)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:8]))
def test_attend(case):
    B, H, Hkv, Nq, d, dtype, page, lengths, rest = case
    per = -(-max(lengths) // page)
    codes, params, order, g = filled(B * per + 1, Hkv, page, d, dtype, seed=sum(lengths))
    table = order[:B * per].reshape(B, per).clone()
    for b, n in enumerate(lengths):  # entries that no token needs
        table[b, -(-n // page):] = -1
    rest = dict(rest)
    if rest.get("slopes"):
        rest["slopes"] = dev([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], torch.float32)
    q = torch.randn(B, H, Nq, d, generator=g, device="cuda").to(dtype)
    a = check_attend(q, codes, params, table, lengths, **rest)
    # a bound on the lengths too low for them, or far too high: the same within rounding
    check_attend(q, codes, params, table, lengths, max_len=1, **rest)
    b = api.cache4_attend(q, codes, params, table, dev(lengths), scale=1.0 / math.sqrt(d), **rest)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), "the same from run to run"


@pytest.mark.parametrize("dtype", [BF, HF])
def test_slots_behind_the_length_do_not_matter(dtype):
    """NaN and infinities in the slots behind a sequence and in front of its window."""
    codes, params, order, g = filled(9, 2, 64, 128, dtype, seed=1)
    table = order[:8].reshape(2, 4).contiguous()
    lengths = [100, 201]
    q = torch.randn(2, 8, 2, 128, generator=g, device="cuda").to(dtype)
    want = check_attend(q, codes, params, table, lengths, window_left=50)
    for b, n in enumerate(lengths):
        for t in list(range(n, 256)) + list(range(0, n - 2 - 50)):
            params[int(table[b, t // 64]), :, :, t % 64] = float("nan") if t % 2 else float("inf")
    got = api.cache4_attend(q, codes, params, table, dev(lengths), scale=1 / math.sqrt(128), window_left=50)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_draft_tokens_that_a_row_does_not_see(dtype):
    """NaN in the slot of a draft's later token, or of one that only earlier rows' windows
    reach: rows that do not see it are as they were."""
    codes, params, order, g = filled(5, 2, 64, 128, dtype, seed=5)
    table = order[:4].reshape(1, 4).contiguous()
    q = torch.randn(1, 8, 3, 128, generator=g, device="cuda").to(dtype)
    want = check_attend(q, codes, params, table, [201], window_left=50)
    for token, clean in ((200, slice(0, 2)), (148, slice(1, 3))):  # rows at 198, 199, 200
        poisoned = params.clone()
        poisoned[int(table[0, token // 64]), :, :, token % 64] = float("nan")
        o, _ = api.cache4_attend(q, codes, poisoned, table, dev([201]), scale=1 / math.sqrt(128), window_left=50)
        assert torch.equal(o[:, :, clean], want[0][:, :, clean])
        assert torch.isnan(o).any(-1).sum() == 8, "the row that sees it"


def test_lengths_near_2_31():
    """The last tokens of the longest sequence that the interface takes: the same as at the end
    of a short one."""
    codes, params, order, g = filled(8, 1, 16, 64, BF, seed=6)
    long = torch.zeros(1, 2**27 - 1, dtype=torch.int32, device="cuda")
    long[0, -8:] = order[:8]
    q = torch.randn(1, 2, 1, 64, generator=g, device="cuda").to(BF)
    kw = dict(window_left=100, max_len=2**31 - 1)
    a = api.cache4_attend(q, codes, params, long, dev([2**31 - 16]), **kw)
    # the same 16 tokens short of a whole step of 32
    short = torch.zeros(1, 2**6 - 1, dtype=torch.int32, device="cuda")
    short[0, -8:] = order[:8]
    b = api.cache4_attend(q, codes, params, short, dev([2**10 - 16]), **kw)
    assert api.fa_get_status() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[1]).all()


def test_one_dominant_key_and_large_scores():
    """Scores of hundreds, where the running maximum moves often, and one that wins."""
    codes, params, order, g = filled(40, 1, 16, 128, BF, seed=2)
    q = (torch.randn(1, 4, 1, 128, generator=g, device="cuda") * 40).to(BF)
    check_attend(q, codes, params, order.reshape(1, 40).contiguous(), [639])
    check_attend(q, codes, params, order.reshape(1, 40).contiguous(), [639], softcap=2.0)


def test_pages_outside_the_cache_are_passed_over_and_noted():
    """Entries outside [0, n_pages), positions outside the table and lengths beyond it."""
    codes, params, order, g = filled(12, 2, 16, 64, BF, seed=3)
    table = order.reshape(2, 6).contiguous()
    table[0, 2], table[1, 0], table[1, 4] = -1, 12, 2**31 - 1
    q = torch.randn(2, 4, 1, 64, generator=g, device="cuda").to(BF)
    check_attend(q, codes, params, table, [90, 96], gone=[(0, 2), (1, 0), (1, 4)], status=FA_ERR_BAD_PAGE)
    o, lse = api.cache4_attend(q, codes, params, table, dev([1000, 2**31 - 1]))  # cut at 96
    assert api.fa_get_status() == FA_ERR_BAD_PAGE
    a, b = api.cache4_attend(q, codes, params, table, dev([96, 96]))
    assert api.fa_get_status() == FA_ERR_BAD_PAGE
    assert torch.equal(o, a) and torch.equal(lse, b)
    k = torch.randn(2, 2, 40, 64, generator=g, device="cuda").to(BF)
    before_c, before_p = codes.clone(), params.clone()
    api.cache4_append(codes, params, k, k, table, dev([24, 90]))  # over page 2 of row 0; past row 1's end
    assert api.fa_get_status() == FA_ERR_BAD_PAGE
    got, _ = api.cache4_read(codes, params, table, dev([24, 90]), 40)
    assert api.fa_get_status() == FA_ERR_BAD_PAGE
    c, s, z = ref4.quantise(k)
    value = (c.float() * s.float() + z.float()).to(BF)
    there = torch.zeros(2, 40, dtype=torch.bool, device="cuda")
    there[0, :8] = there[0, 24:] = True
    there[1, :6] = True
    assert torch.equal(got.transpose(1, 2)[there], value.transpose(1, 2)[there])
    assert (got.transpose(1, 2)[~there] == 0).all()
    held = torch.zeros(12, dtype=torch.bool, device="cuda")
    for b, p in ((0, 1), (0, 3), (1, 5)):
        held[int(table[b, p])] = True
    assert torch.equal(codes[~held], before_c[~held]) and torch.equal(params[~held], before_p[~held])
    api.cache4_append(codes, params, k, k, table, dev([-5, -2**31]), counts=dev([3, 40]))
    assert api.fa_get_status() == FA_ERR_BAD_PAGE
    assert api.fa_get_status() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompt_then_tokens_as_a_model_would(dtype):
    """A prompt through the shaped forward, its keys into the cache, then tokens one by one
    and a draft, each against the cache's codes, and against the shaped forward over the
    values that the cache reads back (which are rounded to the type: another bound)."""
    B, H, Hkv, d, page, n = 2, 8, 2, 64, 32, 75
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda h, m: torch.randn(B, h, m, d, generator=g, device="cuda").to(dtype)  # noqa: E731
    slopes = dev([2.0 ** -(h + 1) for h in range(H)], torch.float32)
    kw = dict(softcap=20.0, slopes=slopes)
    codes, params = api.cache4_empty(B * 4, Hkv, page, d, dtype)
    table = torch.arange(B * 4, device="cuda", dtype=torch.int32).flip(0).reshape(B, 4).contiguous()
    k0, v0 = r(Hkv, n), r(Hkv, n)
    api.forward(r(H, n), k0, v0, causal=True, **kw)
    api.cache4_append(codes, params, k0, v0, table, dev([0, 0]))
    total = n
    for m in (1, 1, 5, 1):
        q = r(H, m)
        api.cache4_append(codes, params, r(Hkv, m), r(Hkv, m), table, dev([total, total]))
        total += m
        check_attend(q, codes, params, table, [total, total], **kw)
        k, v = api.cache4_read(codes, params, table, dev([0, 0]), total)
        full = torch.zeros(B, H, total, d, dtype=dtype, device="cuda")
        full[:, :, -m:] = q
        got = api.forward(full, k, v, causal=True, **kw)
        values, bounds = ref.gradients(full, k, v, full, ref.visible(B, total, True).cuda(), 0.125, 20.0, slopes)
        for a, w, b in zip(got, values, bounds):
            assert ((a.double() - w).abs() <= b).all()
    assert api.fa_get_status() == 0


def test_captured_decode_replays_with_growing_lengths():
    """One captured step (append, then attend) replayed while positions grow in place, beside
    a second captured step of other sequences on another stream."""
    B, H, Hkv, d, page = 2, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(6)
    sets = []
    for s in range(2):
        codes, params, order, _ = filled(64, Hkv, page, d, BF, seed=20 + s)
        st = dict(codes=codes, params=params, table=order.reshape(B, 32).contiguous(), pos=dev([37, 300]),
                  q=torch.zeros(B, H, 1, d, dtype=BF, device="cuda"), k=torch.zeros(B, Hkv, 1, d, dtype=BF, device="cuda"))
        sets.append(st)

    def step(s):
        api.cache4_append(s["codes"], s["params"], s["k"], s["k"], s["table"], s["pos"])
        return api.cache4_attend(s["q"], s["codes"], s["params"], s["table"], s["pos"] + 1)

    graphs, outs = [], []
    for s in sets:
        step(s)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(s))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for s in sets:
            s["q"].copy_(torch.randn(B, H, 1, d, generator=g, device="cuda"))
            s["k"].copy_(torch.randn(B, Hkv, 1, d, generator=g, device="cuda"))
        torch.cuda.synchronize()
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for s, (o, lse) in zip(sets, outs):
            a, b = step(s)
            torch.cuda.synchronize()
            assert torch.equal(o, a) and torch.equal(lse, b)
            s["pos"] += 1
    assert api.fa_get_status() == 0


def test_offsets_beyond_32_bits():
    """Pages whose codes lie past byte 2^32 and row 2^26."""
    Hkv, page, d = 8, 256, 128
    n_pages = 2**32 // (2 * Hkv * page * d // 2) + 3
    codes, params = api.cache4_empty(n_pages, Hkv, page, d)
    table = dev([[n_pages - 1, 0, n_pages - 2]])
    g = torch.Generator(device="cuda").manual_seed(7)
    k = torch.randn(1, Hkv, 600, d, generator=g, device="cuda").to(BF)
    v = torch.randn(1, Hkv, 600, d, generator=g, device="cuda").to(BF)
    api.cache4_append(codes, params, k, v, table, dev([0]))
    got = api.cache4_read(codes, params, table, dev([0]), 600)
    for x, back in zip((k, v), got):
        c, s, z = ref4.quantise(x)
        assert torch.equal(back, (c.float() * s.float() + z.float()).to(BF))
    q = torch.randn(1, 8, 1, d, generator=g, device="cuda").to(BF)
    check_attend(q, codes, params, table, [600])
    del codes
    torch.cuda.empty_cache()
