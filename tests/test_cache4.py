"""The 4-bit cache on the CPU: where a token's rows lie, what the entry points refuse, and the
reference quantiser's own properties."""
import ctypes
import random

import pytest
import torch

import cache4_reference as ref4
from io_aware_attention_flashattention_b200 import _lib, api, build

INT = ctypes.c_int


@pytest.fixture(scope="module")
def libfa():
    build.build_library()
    return _lib.lib()


def _row(lib, table, n_pages, Hkv, page, which, head, token):
    return lib.fa_cache4_row((INT * len(table))(*table), len(table), n_pages, Hkv, page, which, head, token)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_rows_of_tokens(libfa, page):
    """Index into [n_pages, 2, Hkv, page] of every token; -1 without a page."""
    r = random.Random(page)
    Hkv, n_pages = 3, 9
    table = r.sample(range(n_pages), 4) + [-1, n_pages, 2**31 - 1, -2**31]
    where = torch.arange(n_pages * 2 * Hkv * page).reshape(n_pages, 2, Hkv, page)
    for token in list(range(4 * page)) + [4 * page, 8 * page - 1, 8 * page, 2**31 - 1, 2**40, -1, -2**40]:
        which, head = r.randrange(2), r.randrange(Hkv)
        got = _row(libfa, table, n_pages, Hkv, page, which, head, token)
        if 0 <= token < 4 * page:
            assert got == int(where[table[token // page], which, head, token % page])
        else:
            assert got == -1


def test_rows_pass_32_bits(libfa):
    assert _row(libfa, [2**29], 2**30, 8, 256, 1, 7, 255) == ((2**29 * 2 + 1) * 8 + 7) * 256 + 255


def test_row_refusals(libfa):
    t = (INT * 1)(0)
    assert libfa.fa_cache4_row(None, 1, 1, 1, 16, 0, 0, 0) == -1
    for page, which, head in ((24, 0, 0), (8, 0, 0), (512, 0, 0), (16, 2, 0), (16, 0, 1), (16, 0, -1)):
        assert libfa.fa_cache4_row(t, 1, 1, 1, page, which, head, 0) == -1


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_cache_calls_refuse_on_the_host(libfa, suffix):
    P = 0x10000
    for name in ("append", "read"):
        f = getattr(libfa, f"fa_cache4_{name}{suffix}")

        def call(K=P, codes=P, params=P, table=P, pos=P, counts=None, B=2, Hkv=2, n=4, d=64, page=16, n_pages=4,
                 max_pages=2):
            return f(K, P, codes, params, table, pos, counts, B, Hkv, n, d, page, n_pages, max_pages, None)

        assert call(d=96) == 2 and call(page=24) == 2 and call(page=512) == 2 and call(page=8) == 2
        assert call(B=0) == 1 and call(Hkv=0) == 1 and call(n=-1) == 1 and call(n_pages=0) == 1
        assert call(max_pages=0) == 1 and call(max_pages=1 << 27) == 2 and call(n_pages=1 << 31) == 2
        assert call(K=None) == 1 and call(K=P + 8) == 1 and call(codes=P + 4) == 1 and call(params=P + 2) == 1
        assert call(table=None) == 1 and call(table=P + 2) == 1 and call(pos=None) == 1 and call(counts=P + 1) == 1
        assert call(B=1 << 20, n=1 << 20) == 2
        assert call(n=0, K=None) == 0
    f = getattr(libfa, "fa_cache4_attend" + suffix)

    def att(Q=P, codes=P, lengths=P, B=2, H=4, Hkv=2, Nq=1, d=64, page=16, max_pages=4096, max_len=65536, scale=0.1,
            cap=0.0, slopes=None, ws=P, nbytes=1 << 40):
        return f(Q, P, P, codes, P, P, lengths, B, H, Hkv, Nq, d, page, 9, max_pages, max_len, scale, -1, cap, slopes,
                 ws, nbytes, None)

    assert att(d=80) == 2 and att(H=5) == 1 and att(B=0) == 1 and att(Nq=-1) == 1 and att(max_len=-1) == 1
    assert att(scale=0.0) == 1 and att(scale=float("nan")) == 1 and att(cap=-1.0) == 1 and att(cap=1e9) == 2
    assert att(Q=None) == 1 and att(Q=P + 8) == 1 and att(codes=None) == 1 and att(lengths=None) == 1
    assert att(lengths=P + 1) == 1 and att(slopes=P + 2) == 1 and att(page=48) == 2
    need = libfa.fa_cache4_workspace_size(2, 4, 2, 1, 64, 65536, -1)
    assert need > 0 and att(nbytes=need - 1) == 1 and att(ws=None) == 1 and att(ws=P + 8) == 1
    assert att(B=1 << 16, H=1 << 15, Hkv=1) == 2 and att(Nq=1 << 25) == 2
    assert att(B=1 << 10, H=64, Hkv=1, Nq=1 << 15) == 2  # 2^31 rows
    assert att(Nq=0, Q=None) == 0


def test_workspace_size(libfa):
    f = libfa.fa_cache4_workspace_size
    assert f(1, 8, 8, 1, 64, 127, -1) == 0  # short: one piece a sequence
    assert f(1, 8, 8, 1, 64, 0, -1) == 0
    assert f(1, 8, 3, 1, 64, 4096, -1) == 0 and f(1, 8, 8, 1, 96, 4096, -1) == 0
    assert f(8, 32, 8, 4096, 128, 4096, -1) == 0  # many rows: sequences stay whole
    assert f(1, 8, 8, 1, 64, 4096, 2**31 - 1) == f(1, 8, 8, 1, 64, 4096, -1)
    # a window bounds the pieces whatever the length
    assert f(1, 8, 8, 1, 64, 1 << 20, 100) == f(1, 8, 8, 1, 64, 1 << 24, 100)
    assert f(1, 8, 8, 1, 64, 1 << 20, -1) > f(1, 8, 8, 1, 64, 1 << 12, -1) > 0


def test_binding_refuses_wrong_tensors():
    with pytest.raises(ValueError, match="page holds"):
        api.cache4_empty(4, 2, 24, 64, device="cpu")
    with pytest.raises(ValueError, match="64 or 128"):
        api.cache4_empty(4, 2, 16, 96, device="cpu")
    with pytest.raises(TypeError, match="bf16 and f16"):
        api.cache4_empty(4, 2, 16, 64, dtype=torch.float32, device="cpu")
    codes, params = api.cache4_empty(4, 2, 16, 64, device="cpu")
    assert codes.shape == (4, 2, 2, 16, 32) and params.shape == (4, 2, 2, 16, 2)
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    table, pos = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.cache4_append(codes, params, k, k, table, pos)
    with pytest.raises(TypeError, match="bf16 and f16"):
        api.cache4_append(codes, params, k.float(), k.float(), table, pos)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_reference_quantiser(dtype):
    """Values are off by at most half a step and what the rounded step adds at code 15."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(200, 64, generator=g) * torch.logspace(-3, 2, 200)[:, None] + 1).to(dtype)
    code, scale, zero = ref4.quantise(x)
    back = scale.double() * code.double() + zero.double()
    u = torch.finfo(dtype).eps / 2
    step = (x.double().amax(-1) - x.double().amin(-1))[:, None] / 15
    assert ((back - x.double()).abs() <= step * (0.5 + 16 * u)).all()
    flat = torch.full((1, 64), 3.25, dtype=dtype)
    assert ref4.quantise(flat)[0].max() == 0
