"""Attention over prompts whose scores are as large as a call takes: their fp32 steps are then
more than the binary orders between a weight of 1 and the largest fp16 number."""
import pytest
import torch

import paged_kv_cache_154_gb300 as pa

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("dt,q0,k0", [("f16", 59968.0, 2000.0), ("f16", 8192.0, 2000.0),
                                      ("f16", 1024.0, 1024.0), ("bf16", 32768.0, 30464.0),
                                      ("bf16", 8192.0, 2000.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_largest_scores(dt, q0, k0, d):
    """Scores up to the documented 2^27 and 2^30, whose fp32 steps are larger than a weight's
    range, with rises of a few steps from key to key: values of 1 come out as 1. A weight is
    rounded by half a step for the product and not for the sum, the output by another."""
    T, dtype = 700, DT[dt]
    gen = torch.Generator(device="cuda").manual_seed(int(q0) % 997)
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    v = torch.ones((T, 1, d), dtype=dtype, device="cuda")
    for most in (1, 4, 30, 200):
        q, k = (torch.zeros((T, n, d), device="cuda") for n in (2, 1))
        q[..., 0], k[..., 0], q[..., 1] = q0, k0, 16.0
        k[:, 0, 1] = torch.sort(torch.randint(0, most, (T,), generator=gen, device="cuda"))[0]
        k[::7, 0, 1] = 0
        out = torch.empty((T, 2, d), dtype=dtype, device="cuda")
        pa.prompt_attention(out, q.to(dtype), k.to(dtype), v, start, T, 1.0)
        assert pa.device_error() == 0
        eps = torch.finfo(dtype).eps / 2
        assert ((out.double() - 1).abs() <= 2 * eps + eps * eps + T * 5e-9).all()
