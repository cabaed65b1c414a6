"""Slopes that require a gradient: refused where one would be taken, and only there."""
import pytest
import torch

from io_aware_attention_flashattention_b200 import api

BF = torch.bfloat16


def _tensors(device="cpu"):
    g = torch.Generator(device=device).manual_seed(1)
    return [torch.randn(1, 2, 40, 64, generator=g, device=device).to(BF) for _ in range(3)]


def test_refused_under_grad_and_not_without(monkeypatch):
    """With autograd off a call goes on to the kernels with the slopes as they are."""
    q, k, v = _tensors()
    slopes = torch.nn.Parameter(torch.ones(2))
    got = []
    monkeypatch.setattr(api, "forward", lambda *a: (got.append(a[9]), (q, q[..., 0].float()))[1])
    with pytest.raises(ValueError, match="no gradient"):
        api.attention(q, k, v, slopes=slopes)
    assert not got
    with torch.no_grad():
        api.attention(q, k, v, slopes=slopes)
    assert got[0] is slopes


def test_the_function_itself_refuses_the_backward(monkeypatch):
    q, k, v = _tensors()
    slopes = torch.nn.Parameter(torch.ones(2))
    monkeypatch.setattr(api, "forward", lambda *a: (q.clone(), q[..., 0].float()))
    monkeypatch.setattr(api, "backward", lambda *a, **kw: (q, k, v))
    out = api.FlashAttentionFunction.apply(q.clone().requires_grad_(), k, v, True, None, None, None, None, None, slopes)
    with pytest.raises(ValueError, match="no gradient"):
        out.sum().backward()


@pytest.mark.gpu
def test_a_models_own_slopes_in_inference():
    q, k, v = _tensors("cuda")
    slopes = torch.nn.Parameter(torch.tensor([0.5, 0.1], device="cuda"))
    with torch.no_grad():
        o = api.attention(q, k, v, causal=True, slopes=slopes)
    assert torch.equal(o, api.forward(q, k, v, True, slopes=slopes.detach())[0])
