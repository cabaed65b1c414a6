"""Attention with shaped scores, on the CPU: the tests' own 64-bit definition against
autograd and differences, the intervals that the kernels walk against the masks listed
pair by pair, and the refusals of the entry points."""
import ctypes
import math
import random

import pytest
import torch

import score_reference as ref
from io_aware_attention_flashattention_b200 import _lib, build

INT = ctypes.c_int


@pytest.fixture(scope="module")
def libfa():
    build.build_library()
    return _lib.lib()


def _inputs(B, H, Hkv, N, d, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda h: torch.randn(B, h, N, d, generator=g, dtype=torch.float64)  # noqa: E731
    return n(H), n(Hkv), n(Hkv), n(H)


CASES = [
    dict(causal=True, softcap=2.0),
    dict(causal=False, slopes=[0.5, 0.1, 0.0, 2.0]),
    dict(causal=True, window=(3, -1), documents=[[0, 4, 4, 9], [1, 2, 7, 8]], prefix=[[2, 0, 3], [0, 9, -1]]),
    dict(causal=False, window=(2, 1), softcap=1.0, slopes=[1.0, 0.5, 0.25, 0.125], prefix=[3, 0]),
]


def _options(case):
    mask = ref.visible(2, 9, case.get("causal", False), case.get("window", (-1, -1)),
                       case.get("documents"), torch.tensor(case["prefix"]) if "prefix" in case else None)
    slopes = torch.tensor(case["slopes"]) if "slopes" in case else None
    return mask, case.get("softcap"), slopes


@pytest.mark.parametrize("case", CASES)
def test_reference_gradients_match_autograd_and_differences(case):
    q, k, v, do = _inputs(2, 4, 2, 9, 3, 5)
    mask, cap, slopes = _options(case)
    (o, lse, dq, dk, dv), _ = ref.gradients(q, k, v, do, mask, 0.7, cap, slopes)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    out, _ = ref.attention(*leaves, mask, 0.7, cap, slopes)
    live = (lse > -math.inf)[..., None]
    loss = lambda *x: (torch.where(live, ref.attention(*x, mask, 0.7, cap, slopes)[0], 0.0)  # noqa: E731
                       * do).sum()
    assert torch.equal(torch.where(live, out, 0.0), torch.where(live, o, 0.0))
    if live.all():
        for got, want in zip((dq, dk, dv), torch.autograd.grad(loss(*leaves), leaves)):
            assert (got - want).abs().max() < 1e-12
    rng = random.Random(3)
    for n, grad in enumerate((dq, dk, dv)):
        for _ in range(12):
            at = tuple(rng.randrange(s) for s in grad.shape)
            h = 1e-6
            side = []
            for sign in (1, -1):
                x = [t.clone() for t in (q, k, v)]
                x[n][at] += sign * h
                side.append(loss(*x))
            assert abs((side[0] - side[1]) / (2 * h) - grad[at]) < 1e-7


def _span(lib, what, index, N, causal, window, docs, prefix):
    a = None if docs is None else (INT * len(docs))(*docs)
    p = None if prefix is None else (INT * len(prefix))(*prefix)
    lo, hi = INT(-5), INT(-5)
    st = lib.fa_score_span(a, 0 if docs is None else len(docs) - 1, p, N, int(causal), *window, what,
                           index, ctypes.addressof(lo), ctypes.addressof(hi))
    assert st == 0
    return lo.value, hi.value


@pytest.mark.parametrize("seed", range(40))
def test_intervals_are_the_mask(libfa, seed):
    """Keys of a query and queries of a key are the mask's rows and columns, and the tiles
    that are walked hold all of them, for ascending offsets, empty documents and padding."""
    r = random.Random(seed)
    N = r.choice([1, 2, 5, 127, 128, 129, 300, 511])
    causal = r.random() < 0.6
    window = (r.choice([-1, -1, 0, 1, r.randint(0, N + 3)]), r.choice([-1, -1, 0, r.randint(0, N + 3)]))
    M = r.choice([0, 1, 2, 7])
    docs = sorted(r.randint(0, N) for _ in range(M + 1)) if M else None
    prefix = [r.choice([0, 1, -3, r.randint(0, N), 2**31 - 1]) for _ in range(max(1, M))] if r.random() < .5 else None
    mask = ref.visible(1, N, causal, window, None if docs is None else [docs],
                       None if prefix is None else torch.tensor([prefix]))[0]
    for i in range(N):
        for what, line in ((0, mask[i]), (1, mask[:, i])):
            lo, hi = _span(libfa, what, i, N, causal, window, docs, prefix)
            assert line.nonzero().flatten().tolist() == list(range(lo, hi)), (what, i)
    for r0 in range(0, N, 128):
        for what, lines in ((2, mask[r0:r0 + 128]), (3, mask[:, r0:r0 + 128].T)):
            lo, hi = _span(libfa, what, r0, N, causal, window, docs, prefix)
            hit = {int(x) // 128 for x in lines.any(0).nonzero()}
            assert hit <= set(range(lo, hi))
            assert not hit or (lo, hi) == (min(hit), max(hit) + 1)


def test_intervals_stay_inside_for_any_offsets(libfa):
    """Offsets that do not ascend or leave [0, N] give some interval inside the row."""
    r = random.Random(1)
    for _ in range(400):
        N = r.choice([1, 100, 128, 500])
        wild = lambda: r.choice([0, N, -1, r.randint(-N, 2 * N), 2**31 - 1, -2**31])  # noqa: E731
        docs = [wild() for _ in range(r.randint(2, 9))]
        prefix = [wild() for _ in range(len(docs) - 1)] if r.random() < 0.5 else None
        window = (r.choice([-1, 0, 50, 2**31 - 1]), r.choice([-1, 0, 50]))
        for what in range(4):
            index = r.randrange(N)
            lo, hi = _span(libfa, what, index, N, r.random() < .5, window, docs, prefix)
            top = N if what < 2 else (N + 127) // 128
            assert hi <= lo or (0 <= lo and hi <= top), (what, index, N, docs, lo, hi)


def test_span_refusals(libfa):
    lo = INT(0)
    at = ctypes.addressof(lo)
    f = libfa.fa_score_span
    assert f(None, 0, None, 0, 0, -1, -1, 0, 0, at, at) == 1
    assert f(None, 0, None, 8, 0, -1, -1, 4, 0, at, at) == 1
    assert f(None, 0, None, 8, 0, -1, -1, 0, 8, at, at) == 1
    assert f(None, 0, None, 8, 2, -1, -1, 0, 0, at, at) == 1
    assert f((INT * 2)(0, 8), 0, None, 8, 0, -1, -1, 0, 0, at, at) == 1
    assert f(None, 0, None, 8, 0, -1, -1, 0, 0, None, at) == 1


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_scored_calls_refuse_on_the_host(libfa, suffix):
    P = 0x10000
    f = getattr(libfa, "fa_forward_scored" + suffix)

    def fwd(B=1, H=4, Hkv=2, N=128, d=64, scale=0.125, causal=1, cap=0.0, slopes=None, docs=None, n=0, pre=None,
            q=P):
        return f(q, P, P, P, P, B, H, Hkv, N, d, scale, causal, -1, -1, cap, slopes, docs, n, pre, None)

    assert fwd(H=4, Hkv=3) == 1 and fwd(Hkv=0) == 1 and fwd(Hkv=8) == 1
    assert fwd(d=96) == 2 and fwd(causal=2) == 1 and fwd(q=None) == 1 and fwd(q=P + 2) == 1
    assert fwd(cap=-1.0) == 1 and fwd(cap=float("nan")) == 1 and fwd(cap=float("inf")) == 1
    assert fwd(cap=1e-6) == 2 and fwd(cap=1e9) == 2  # scale / cap outside [2^-24, 2^12]
    assert fwd(docs=P, n=0) == 1 and fwd(docs=P + 2, n=1) == 1 and fwd(slopes=P + 1) == 1
    assert fwd(pre=P + 3) == 1
    assert fwd(N=0, q=None) == 0 and fwd(N=0, H=4, Hkv=3) == 1
    b = getattr(libfa, "fa_backward_scored" + suffix)
    ws = libfa.fa_backward_workspace_size(1, 4, 384, 64)

    def bwd(Hkv=2, cap=0.0, nbytes=ws, w=P, dq=P):
        return b(P, P, P, P, P, P, dq, P, P, 1, 4, Hkv, 384, 64, 0.125, 1, -1, -1, cap, None, None, 0, None, w,
                 nbytes, None)

    assert bwd(Hkv=3) == 1 and bwd(cap=-2.0) == 1 and bwd(nbytes=ws - 1) == 1 and bwd(w=None) == 1
    assert bwd(dq=None) == 1


def test_scored_workspace_size(libfa):
    f, base = libfa.fa_backward_scored_workspace_size, libfa.fa_backward_workspace_size
    assert f(3, 8, 3, 1531, 64) == 0 and f(3, 8, 2, 1531, 96) == 0 and f(1, 8, 2, 0, 64) == 0
    # 72 key tiles of 4 heads each: two waves of 148 take 4 segments each, dK and dV partials
    # of 128 rows in fp32, and a counter per tile
    assert f(3, 8, 2, 1531, 64) == base(3, 8, 1531, 64) + 72 * 4 * 2 * 128 * 64 * 4 + 512
    assert f(2, 16, 4, 4096, 128) == base(2, 16, 4096, 128)  # 256 tiles: whole
    # one query tile of 6 heads: 3 segments of two steps
    assert f(1, 6, 1, 128, 64) == base(1, 6, 128, 64) + 3 * 2 * 128 * 64 * 4 + 256
    assert f(1, 2, 1, 128, 64) == base(1, 2, 128, 64)  # two steps: whole
    assert f(1, 8, 8, 128, 64) == base(1, 8, 128, 64)  # nothing to part


def test_binding_refuses_what_does_not_combine():
    from io_aware_attention_flashattention_b200 import api

    q = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="do not combine"):
        api.forward(q, k, k, dropout=(0.1, 1, 0))
    with pytest.raises(ValueError, match="do not combine"):
        api.forward(q, q, q, block_mask=torch.ones(1, 1, dtype=torch.uint8), softcap=5.0)
    with pytest.raises(TypeError, match="bf16 and f16"):
        api.forward(q.float(), k.float(), k.float())
    with pytest.raises(ValueError, match="evenly"):
        api.forward(q, torch.zeros(1, 3, 8, 64, dtype=torch.bfloat16), q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.forward(q, k, k)
    with pytest.raises(ValueError, match="no gradient"):
        api.attention(q, k, k, slopes=torch.ones(4, requires_grad=True))
    with pytest.raises(ValueError, match="offsets"):
        api._score(1, 4, None, None, torch.zeros(3, dtype=torch.int32), None)


def test_binding_holds_windows_to_32_bits():
    from io_aware_attention_flashattention_b200 import api

    assert api._window((2**40, 2**32)) == (2**31 - 1, 2**31 - 1)
    assert api._window((-2**40, 5)) == (-1, 5) and api._window(None) == (-1, -1)
