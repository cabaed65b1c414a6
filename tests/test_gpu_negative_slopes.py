"""Distance biases of either sign: negative slopes raise the scores of far keys, so the largest
scores lie at the far end of a row."""
import math

import pytest
import torch

import score_reference as ref
from io_aware_attention_flashattention_b200 import api
from test_gpu_cache4 import check_attend, dev, filled
from test_gpu_score import check, make, run

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("B,H,Hkv,N,d,dtype,causal,window,softcap", [
    (1, 4, 2, 500, 64, BF, True, (-1, -1), None),
    (2, 4, 4, 300, 128, HF, False, (-1, -1), None),
    (1, 4, 1, 400, 128, BF, True, (100, -1), 20.0),
    (1, 4, 2, 260, 64, HF, False, (70, 90), 15.0),
    (1, 4, 4, 1, 64, BF, True, (-1, -1), None),
])
def test_forward_and_backward(B, H, Hkv, N, d, dtype, causal, window, softcap):
    q, k, v, do = make(B, H, Hkv, N, d, dtype, seed=N)
    slopes = torch.tensor([-0.5, -0.03, 0.0, 0.25], device="cuda")
    scale = 1 / math.sqrt(d)
    got = run(q, k, v, do, scale, causal, window, dict(softcap=softcap, slopes=slopes))
    check(got, q, k, v, do, ref.visible(B, N, causal, window), scale, softcap, slopes)


@pytest.mark.parametrize("dtype,Nq,window_left,softcap", [(BF, 1, -1, None), (HF, 4, 200, 10.0)])
def test_over_the_cache(dtype, Nq, window_left, softcap):
    codes, params, order, g = filled(40, 2, 32, 128, dtype, seed=Nq)
    table = order.reshape(2, 20).contiguous()
    q = torch.randn(2, 4, Nq, 128, generator=g, device="cuda").to(dtype)
    slopes = dev([-0.4, -0.01, 0.0, 0.3], torch.float32)
    check_attend(q, codes, params, table, [77, 600], window_left=window_left, softcap=softcap, slopes=slopes)
    assert api.fa_get_status() == 0
