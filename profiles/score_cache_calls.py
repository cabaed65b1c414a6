"""One call of each main kernel of the shaped passes and the 4-bit cache, twice (the second round is
the one to profile): inputs larger than L2, 1.2 GB on the device."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from io_aware_attention_flashattention_b200 import api  # noqa: E402

BF = torch.bfloat16
g = torch.Generator(device="cuda").manual_seed(1)


def r(*shape):
    return torch.randn(*shape, device="cuda", generator=g).to(BF)


q1, k1, v1 = r(2, 16, 8192, 128), r(2, 8, 8192, 128), r(2, 8, 8192, 128)
q2, k2, v2, do2 = r(2, 16, 4096, 128), r(2, 4, 4096, 128), r(2, 4, 4096, 128), r(2, 16, 4096, 128)
codes, params = api.cache4_empty(64 * 128, 8, 64, 128)
codes.random_(0, 256, generator=g)
params[..., 0] = (torch.rand(params.shape[:-1], device="cuda", generator=g) * 0.3 + 0.05).to(BF)
params[..., 1] = -2.5
table = torch.randperm(64 * 128, device="cuda", generator=g).to(torch.int32).reshape(64, 128)
lengths = torch.randint(2048, 8193, (64,), device="cuda", generator=g).to(torch.int32)
q3, k4, v4 = r(64, 32, 1, 128), r(16, 8, 2048, 128), r(16, 8, 2048, 128)
first = table[:16].contiguous()
zero = torch.zeros(16, dtype=torch.int32, device="cuda")
o2, lse2 = api.forward(q2, k2, v2, causal=True, softcap=50.0)
torch.cuda.synchronize()
for _ in range(2):
    api.forward(q1, k1, v1, causal=True, window=(1024, -1), softcap=30.0)
    api.backward(q2, k2, v2, o2, lse2, do2, causal=True, softcap=50.0)
    api.cache4_attend(q3, codes, params, table, lengths, softcap=50.0, max_len=8192)
    api.cache4_append(codes, params, k4, v4, first, zero)
    api.cache4_read(codes, params, first, zero, 2048)
torch.cuda.synchronize()
assert api.fa_get_status() == 0
