"""Attention over prompts whose weights are far below the largest one, which fp16 cannot hold
beside it without care: a sink at the first token that takes nearly all of the weight and whose
value is zero, so that the output is what the others give.

Tolerance, derived before the first run. Relative to the reference of a row, which is at most
its largest weight, weights are held in fp16 2^8 above: off by half a step, 2^-11 of themselves,
and from 2^-14 / 2^8 down by half a subnormal step, 2^-25 / 2^8 = 2^-33 of the largest weight.
bf16 holds them to 2^-8 of themselves. Scores, exponentials and sums as in the other tests of
prompt attention: scores up to 30 in magnitude, off by (d + 4) 2^-24 of them, 2.4e-4 of a
weight, and 2^-21. Sums of the products lose up to 5e-9 a key in the tensor cores. All of it
acts on the sum of p |v|, and the output is off by half a step of its own, in fp16 at least half
of a subnormal step."""
import numpy as np
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


def sink(T, H, d, dtype, gap, at=0, size=1024.0):
    """Rows whose key `at` scores `gap` above the others' mean, and has a value of 0; the others'
    scores spread by 0.5, their values lie around `size`, for outputs that fp16 holds."""
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    q, k = (torch.randn((T, n, d), device="cuda", generator=gen) * 0.7 for n in (H, 1))
    k[..., 0] = 0
    q[..., 0] = 4.0
    k[at, 0] = 0
    k[at, 0, 0] = gap * d ** 0.5 / 4.0
    v = (torch.rand((T, 1, d), device="cuda", generator=gen) + 0.5) * size
    v[at] = 0
    return q.to(dtype), k.to(dtype), v.to(dtype)


def check_rows(out, q, k, v, rows, scale, dtype, short):
    """short: the part of a sum that the tensor cores may cut off."""
    eps = torch.finfo(dtype).eps / 2
    for row in rows:
        s = (q[row].double() @ k[:row + 1, 0].double().t()) * scale
        p, x = torch.softmax(s, -1), v[:row + 1, 0].double()
        want, size = p @ x, p @ x.abs()
        tol = (eps + 2.4e-4 + 2.0 ** -21 + short) * size * (1 + eps) + eps * want.abs()
        if dtype == torch.float16:
            tol += 2.0 ** -25 + 2.0 ** -33 * (p.amax(-1, keepdim=True) * x.abs().sum(0))
        got = out[row].double()
        off = ((got - want).abs() / tol).max().item()
        assert torch.isfinite(got).all() and off <= 1, (row, off)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap", [10.0, 16.0, 18.0])
def test_sink_without_a_value(dt, d, gap):
    """What the other tokens give, e^-10 to e^-18 of the sink each, is neither cut nor lost."""
    T, dtype = 4096, DT[dt]
    q, k, v = sink(T, 2, d, dtype, gap)
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pa.prompt_attention(out, q, k, v, start, T, d ** -0.5)
    assert pa.device_error() == 0
    check_rows(out, q, k, v, (1, 31, 128, 500, 1023, 2047, 3333, T - 1), d ** -0.5, dtype,
               5e-9 * T)


@pytest.mark.parametrize("at", [40, 100, 130, 9000])
def test_sink_that_comes_later(at):
    """The reference moves when the sink comes: in a tile's first half, its second, in a later
    tile, behind a span of kept sums. Earlier rows do not know it."""
    T, d, dtype = 10000, 64, torch.float16
    q, k, v = sink(T, 2, d, dtype, 18.0, at)
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ws = torch.full((pa.prompt_attention_workspace_size(d, T),), 255, dtype=torch.uint8,
                    device="cuda")
    out = torch.empty_like(q)
    pa.prompt_attention(out, q, k, v, start, T, d ** -0.5, ws)
    assert pa.device_error() == 0
    check_rows(out, q, k, v, (at - 1, at, at + 1, at + 300, 9500, T - 1), d ** -0.5, dtype, 6.1e-5)


def rises(T, d, keys, dtype):
    """Keys of which those named score so many binary orders above the rest (channel 0 alone);
    the rest score 0."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, k = (torch.zeros((T, n, d), device="cuda") for n in (2, 1))
    v = torch.randn((T, 1, d), device="cuda", generator=gen)
    q[..., 0] = 8.0
    for key, orders in keys.items():
        k[key, 0, 0] = orders / 8.0             # with a scale of ln 2, below
    return q.to(dtype), k.to(dtype), v.to(dtype)


@pytest.mark.parametrize("dt,orders", [("f16", (6.75, 7.0, 7.25, 8.0, 15.0)),
                                       ("bf16", (14.75, 15.0, 15.25, 16.0, 40.0))])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_on_either_side_of_the_bounds(dt, orders, d):
    """High keys in second halves of several tiles, at and about the rise from which the
    reference moves, and first halves whose weights' sum is just below and just above 2^15 (one
    key of nearly 2^15 above 63 others, two of half of it, 64 of a 64th). fp16: the others'
    weights are 2^8 each."""
    T, dtype = 700, DT[dt]
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lift = 8.0 if dt == "f16" else 0.0
    cases = [{key: r for key in second} for r in orders
             for second in ((70,), (127, 200, 255), (500, 501, 502))]
    for below in (-0.0625, 0.0, 0.0625):
        top = 15.0 - lift + below
        cases += [{130: top}, {140: top - 1, 150: top - 1},
                  {key: top - 6 for key in range(128, 192)}]
    for keys in cases:
        q, k, v = rises(T, d, keys, dtype)
        out = torch.empty_like(q)
        pa.prompt_attention(out, q, k, v, start, T, float(np.log(2.0)))
        assert pa.device_error() == 0
        check_rows(out, q, k, v, (39, 69, 70, 127, 128, 135, 160, 191, 255, 256, 501, T - 1),
                   float(np.log(2.0)), dtype, 5e-9 * T)
