"""Calls of the attention half at the edges of what they document: tiles that follow one another in a CTA, values that are
not finite, batches without a token, weights far below the largest, memory that overlaps.  64-bit forms: attn_ref."""
import math

import pytest
import torch

import attn_ref as ref
import ternary_weight_moe_forward_b200 as tw

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def ints(r, n, k):
    return torch.clamp(torch.round(r(n, k) * 40), -127, 127).to(torch.int8)


def linear_ref(x, w, alpha, bias=None, resid=None):
    """Codes, exact sums, and the roundings in the documented order: the result to the bit."""
    amax = x.float().abs().amax(1, keepdim=True)
    q = torch.round(x.float() * (torch.full_like(amax, 127.0) / amax)).clamp(-127, 127)
    q = torch.where(amax > 0, q, torch.zeros_like(q))
    acc = (q.double() @ w.double().t()).float()
    y = acc * (alpha * (amax / torch.full_like(amax, 127.0)))
    if bias is not None:
        y = y + bias
    return y if resid is None else resid + y


# Sizes that lead to tiles of 160, 192 and 224 columns, more of them than SMs: some or all warps of a CTA store an odd number
# of pieces of 32 columns per tile
@pytest.mark.parametrize("T,N", [(2048, 2560), (3431, 1288), (2000, 5120), (3431, 1648), (4096, 2560), (2000, 8192)])
@pytest.mark.parametrize("K", [16, 128, 256])
def test_linear_tiles_that_follow_one_another(T, N, K):
    r = gen(T + N + K)
    x, w, al = r(T, K).to(BF16), ints(r, N, K), r(N).abs() * 0.01
    want = linear_ref(x, w, al).to(BF16)
    for _ in range(20):
        assert torch.equal(tw.int8_linear(x, w, al, out_dtype=BF16), want)
