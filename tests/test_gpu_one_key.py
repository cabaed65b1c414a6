"""Masks that leave every row one key: its weight is 1 whatever the scores, so dQ and dK are 0
exactly and dV is dO, through every call that takes such a mask."""
import pytest
import torch

from io_aware_attention_flashattention_b200 import api
from test_gpu_score import make

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def check(v, do, o, grads):
    torch.cuda.synchronize()
    assert api.fa_get_status() == 0
    assert torch.equal(o, v) and torch.equal(grads[2], do)
    assert (grads[0] == 0).all() and (grads[1] == 0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,causal,window", [(300, False, (0, 0)), (300, True, (0, -1)), (300, True, (0, 7)),
                                             (129, True, (0, 0)), (1, False, None), (1, True, (5, 5)),
                                             (1, False, (0, 0))])
def test_through_the_convenience_calls(dtype, d, N, causal, window):
    q, k, v, do = make(2, 3, 3, N, d, dtype, seed=N)
    o, lse = api.forward(q, k, v, causal, window=window)
    check(v, do, o, api.backward(q, k, v, o, lse, do, causal, window=window))
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    out = api.attention(*leaves, causal, window=window)
    out.backward(do)
    check(v, do, out, [x.grad for x in leaves])


@pytest.mark.parametrize("call", ["fa_backward", "fa_backward_f16", "fa_backward_masked", "fa_backward_masked_causal",
                                  "fa_backward_noalloc"])
def test_through_the_entry_points(call):
    dtype = HF if call.endswith("f16") else BF
    masked = "masked" in call
    q, k, v, do = make(2, 3, 3, 260 if masked else 1, 64, dtype, seed=7)
    window, causal = (0, -1 if call.endswith("causal") else 0) if masked else None, call.endswith("causal")
    o, lse = api.forward(q, k, v, causal, window=window)
    grads = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    ws = api.workspace_for(q).fill_(0xFF)
    if masked:
        api.fa_backward_masked(q, k, v, o, do, lse, *grads, 0.125, causal, ws, window)
    elif call == "fa_backward_noalloc":
        api.fa_backward_noalloc(q, k, v, o, do, lse, *grads, 0.125, False)
    else:
        getattr(api, call)(q, k, v, o, do, lse, *grads, 0.125, False, ws)
    check(v, do, o, grads)


def test_an_empty_key_and_dropout_keep_their_own_calls():
    """A block mask that drops the only key leaves a row without keys, not with one; dropout of
    the only key leaves its output 0."""
    q, k, v, do = make(1, 1, 1, 1, 64, BF, seed=1)
    none = torch.zeros(1, 1, dtype=torch.uint8, device="cuda")
    o, lse = api.forward(q, k, v, block_mask=none)
    grads = api.backward(q, k, v, o, lse, do, block_mask=none)
    assert (o == 0).all() and (lse == -float("inf")).all() and all((x == 0).all() for x in grads)
    for offset in range(8):
        drop = (0.5, 3, offset)
        o, lse = api.forward(q, k, v, dropout=drop)
        dq, dk, dv = api.backward(q, k, v, o, lse, do, dropout=drop)
        kept = bool((o != 0).any())
        assert torch.equal(o, 2 * v if kept else 0 * v) and torch.equal(dv, 2 * do if kept else 0 * do)
