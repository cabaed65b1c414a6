"""Head-sharded calls whose K/V heads are shared by groups of query heads: head counts that do not
divide are refused before any shard runs, and valid ones are cut by K/V heads."""
import itertools

import pytest
import torch

import score_reference as ref
from io_aware_attention_flashattention_b200 import api, sharded

BF, HF = torch.bfloat16, torch.float16


def _uneven(B, H, Hkv, n, monkeypatch):
    """Both calls raise, and no shard was handed to the kernels."""
    ran = []
    monkeypatch.setattr(api, "forward", lambda *a, **kw: ran.append("forward"))
    monkeypatch.setattr(api, "backward", lambda *a, **kw: ran.append("backward"))
    q, k = torch.zeros(B, H, 4, 64, dtype=BF), torch.zeros(B, Hkv, 4, 64, dtype=BF)
    lse, devices = torch.zeros(B, H, 4), ["cuda:0"] * n
    with pytest.raises(ValueError, match="cannot share"):
        sharded.forward_sharded(q, k, k, devices)
    with pytest.raises(ValueError, match="cannot share"):
        sharded.backward_sharded(q, k, k, q, lse, q, devices)
    assert not ran


@pytest.mark.parametrize("H,Hkv,n", [(4, 3, 2), (6, 4, 2), (8, 6, 2), (4, 3, 1), (2, 4, 2), (4, 0, 2), (16, 12, 8)])
@pytest.mark.parametrize("B", [1, 3])
def test_head_counts_that_do_not_divide_are_refused(B, H, Hkv, n, monkeypatch):
    _uneven(B, H, Hkv, n, monkeypatch)


def test_shapes_of_k_and_v_are_checked_before_any_shard():
    t = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    q = t(2, 4, 8, 64)
    for k, v in ((t(2, 4, 8, 64), t(2, 2, 8, 64)), (t(1, 8, 8, 64), t(1, 8, 8, 64)),
                 (t(2, 4, 9, 64), t(2, 4, 9, 64)), (t(2, 4, 8, 128), t(2, 4, 8, 128))):
        with pytest.raises(ValueError, match="k and v must be"):
            sharded.forward_sharded(q, k, v, ["cuda:0", "cuda:0"])


def test_a_shard_holds_the_query_heads_of_its_kv_heads():
    for B, Hkv, group, n in itertools.product((1, 2, 3), (1, 2, 3, 5), (1, 2, 4), (1, 2, 3, 8)):
        H = group * Hkv
        q, k = torch.zeros(B, H, 1, 64), torch.zeros(B, Hkv, 1, 64)
        seen_q, seen_kv = [], []
        for (a, b), (ka, kb), _ in sharded._shards(q, k, k, ["cuda:0"] * n):
            assert b > a and kb > ka
            for i in range(a, b):
                batch, h = divmod(i, H)
                assert ka + (i - a) // ((b - a) // (kb - ka)) == batch * Hkv + h // group
            seen_q += range(a, b)
            seen_kv += range(ka, kb)
        assert seen_q == list(range(B * H)) and seen_kv == list(range(B * Hkv))
        if group == 1:
            want = [r for r in sharded.shard_ranges(B * H, n) if r[0] < r[1]]
            assert [s[0] for s in sharded._shards(q, k, k, ["cuda:0"] * n)] == want


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,N,d,dtype,causal,n", [
    (1, 4, 2, 100, 64, BF, True, 2), (2, 6, 3, 77, 128, HF, False, 4), (1, 8, 2, 300, 64, BF, True, 2),
    (2, 4, 1, 200, 128, HF, True, 3), (1, 4, 2, 1, 64, BF, True, 1)])
def test_shared_heads_match_the_unsharded_call(B, H, Hkv, N, d, dtype, causal, n):
    """O and LSE bit for bit; dK and dV too where one tile of keys is run whole in both (else a
    group may be parted otherwise), and all gradients within the bounds of their roundings."""
    g = torch.Generator(device="cuda").manual_seed(N)
    t = lambda h: torch.randn(B, h, N, d, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v, do = t(H), t(Hkv), t(Hkv), t(H)
    devices = [f"cuda:{i % torch.cuda.device_count()}" for i in range(n)]
    o, lse = sharded.forward_sharded(q, k, v, devices, causal)
    grads = sharded.backward_sharded(q, k, v, o, lse, do, devices, causal)
    o1, lse1 = api.forward(q, k, v, causal)
    whole = api.backward(q, k, v, o1, lse1, do, causal)
    torch.cuda.synchronize()
    assert api.fa_get_status() == 0
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    if N <= 128 and H // Hkv == 2:
        assert torch.equal(grads[1], whole[1]) and torch.equal(grads[2], whole[2])
    values, bounds = ref.gradients(q, k, v, do, ref.visible(B, N, causal).cuda(), d ** -0.5)
    for got, want, bound in zip(grads, values[2:], bounds[2:]):
        assert got.shape == want.shape and ((got.double() - want).abs() <= bound).all()
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    out = sharded.attention_sharded(*leaves, devices, causal)
    out.backward(do)
    assert torch.equal(out, o)
    assert torch.equal(leaves[1].grad, grads[1]) and torch.equal(leaves[2].grad, grads[2])


def test_a_piece_starts_on_16_bytes():
    lse = torch.arange(5 * 77, dtype=torch.float32).reshape(1, 5, 77)
    for a, b in sharded.shard_ranges(5, 3):
        x = sharded._piece(lse, a, b, torch.device("cpu"))
        assert x.data_ptr() % 16 == 0 and torch.equal(x[0], lse[0, a:b])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [77, 129, 1])
def test_rows_of_any_length_on_the_tensors_own_device(N):
    q, k, v, do = (torch.randn(1, 5, N, 64, device="cuda").to(BF) for _ in range(4))
    o, lse = api.forward(q, k, v, True)
    got = sharded.backward_sharded(q, k, v, o, lse, do, ["cuda:0"] * 3, True)
    want = api.backward(q, k, v, o, lse, do, True)
    torch.cuda.synchronize()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
