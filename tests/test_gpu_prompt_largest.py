"""The longest prompt that a call of prompt attention takes, 2^22 tokens.

Tolerance, derived before the first run, as for the sums of long prompts: values lie between 0.5
and 1.5, so that a sum of p |v| is the output itself; weights are rounded by half a step and the
output by another, a span of 8192 keys loses at most 6.1e-5 of its sum in the tensor cores, and
fp16 weights (2^-33 of the largest one of 2^22 keys whose scores spread by 0.7 at most) nothing
beside that. The mean over the d columns also holds the rounding of the outputs, around 1: a step
of eps / sqrt(12 d) a standard deviation of it, 4 of them."""
import pytest
import torch

import paged_kv_cache_154_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)], ids=str)
def test_longest_prompt(dtype, d):
    T = 1 << 22
    gen = torch.Generator(device="cuda").manual_seed(d)
    q, k = ((torch.randn((T, 1, d), device="cuda", generator=gen) * 0.3).to(dtype)
            for _ in range(2))
    v = (torch.rand((T, 1, d), device="cuda", generator=gen) + 0.5).to(dtype)
    ws = torch.full((pa.prompt_attention_workspace_size(d, T),), 255, dtype=torch.uint8,
                    device="cuda")
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    pa.prompt_attention(out, q, k, v, start, T, d ** -0.5, ws)
    assert pa.device_error() == 0
    assert torch.isfinite(out).all()
    eps = torch.finfo(dtype).eps
    for row in (0, 1, 127, 8191, 8192, 1 << 16, (1 << 21) + 5, T - 257, T - 1):
        s = (k[:row + 1, 0].double() @ q[row, 0].double()) * d ** -0.5
        want = torch.softmax(s, -1) @ v[:row + 1, 0].double()
        off = (out[row, 0].double() - want) / want
        assert off.abs().max().item() < eps + 6.1e-5 + eps * eps
        if row >= 8191:     # weights' roundings, of either sign, cancel over that many keys
            assert abs(off.mean().item()) < 6.1e-5 + 4 * eps / (12 * d) ** 0.5
