"""INT4 decode where its number formats come to their ends: values near the
largest and the smallest fp32 numbers, weights far below a row's largest, and
shares of hundreds of blocks. Tolerances are derived beside each test; those of
logits and weights are test_gpu_int4's."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from gpu_harness import half_ulp
from oracle import compressed as ref
from test_gpu_int4 import REL, decode, new_cache, sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def rescaled(cache, tables, lens, factor):
    """V of every context times `factor` (a power of two for each), by its scales: what an
    append of so scaled rows stores, its quantiser's numbers being relative to the scale."""
    for s, L in enumerate(lens):
        live = torch.from_numpy(tables[s, :(L + 15) // 16]).long().cuda()
        cache.v_scale[live] *= factor


# contexts that a warp holds whole, and contexts cut into pieces; one query row and several
SHAPES = [([200, 17], [1, 1], 8, 2, 128), ([200, 17], [5, 2], 16, 2, 64),
          ([5000, 40, 900], [1, 1, 1], 32, 8, 128), ([5000, 40, 900], [3, 1, 2], 16, 2, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{max(s[0])}_run{max(s[1])}_d{s[4]}")
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("log2", [100, 110, 122, -60, -110, -121])
def test_values_near_the_ends_of_fp32(shape, out_dtype, log2):
    """A group's range only has to be finite in fp32; rows of 2^122 times normal
    numbers have ranges up to 2^126, those of 2^-121 scales near 2^-123. The error is
    relative to the largest value, as ever, and a few of the smallest fp32 numbers more:
    an output below 2^-126 is rounded to a multiple of 2^-149 by the piece, by each of
    its (at most 400) pieces' parts and at the end: 2^-140 in all."""
    lens, runs, H, Hkv, d = shape
    cache, tables, qsl, q = sequences(41, lens, runs, H, Hkv, d, torch.bfloat16, junk=False)
    rescaled(cache, tables, lens, 2.0 ** log2)
    got = decode(cache, tables, lens, runs, qsl, q, out_dtype, d ** -0.5)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    k, v = ref.cache_values(cache)
    assert np.abs(v[np.isfinite(v)]).max() < 2.0 ** 127
    want = ref.attend(q.double().numpy(), k, v, tables, lens, qsl, d ** -0.5)
    top = max(np.abs(ref.tokens_of(v, tables[s], L, g)).max()
              for s, L in enumerate(lens) for g in range(Hkv))
    tol = REL * top + 2.0 ** -140
    if out_dtype != torch.float32:
        # below bf16's smallest normal number its steps are 2^-133
        tol = tol + np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(want), 1e-300))) - 8,
                                       -134))
    out = got.double().cpu().numpy()
    assert np.isfinite(out).all()
    assert (np.abs(out - want) <= tol).all(), np.abs(out - want).max() / top


@pytest.mark.parametrize("factor", [1e33, 2e36, 1e-36])
def test_rows_appended_near_the_ends_of_fp32(factor):
    """The same through the append, whose quantiser has a branch of its own for such rows."""
    L, H, d, nb = 700, 2, 64, 50
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn((L, H, d), generator=gen) for _ in range(2))
    k, v = k.bfloat16(), (v * factor).bfloat16()
    cache = new_cache(nb, H, d)
    table = np.random.default_rng(1).permutation(nb)[:(L + 15) // 16].astype(np.int32)[None]
    t = np.arange(L)
    slots = torch.from_numpy(table[0, t // 16].astype(np.int64) * 16 + t % 16).cuda()
    pa.append_kv(k.cuda(), v.cuda(), cache.k, cache.v, slots, nb, cache.k_scale, cache.v_scale,
                 cache.k_zp, cache.v_zp)
    q = torch.randn((1, 8, d), generator=gen).bfloat16()
    qsl = np.arange(2, dtype=np.int32)
    got = decode(cache, table, [L], [1], qsl, q, torch.float32, 0.125).double().cpu().numpy()
    kv, vv = ref.cache_values(cache)
    held = ref.values_int4(*ref.quantise_int4(v.float().numpy()))
    for g in range(H):
        assert np.array_equal(ref.tokens_of(vv, table[0], L, g), held[:, g])
    want = ref.attend(q.double().numpy(), kv, vv, table, [L], qsl, 0.125)
    assert np.isfinite(got).all()
    assert np.abs(got - want).max() <= REL * np.abs(held).max()


def test_pieces_of_rows_that_see_nothing_of_them():
    """Query rows that see no token of a late piece, with values whose sums would not be
    finite: such a piece counts for nothing."""
    lens, runs, H, Hkv, d = [2000, 1990], [40, 16], 2, 1, 128
    cache, tables, qsl, q = sequences(43, lens, runs, H, Hkv, d, torch.bfloat16)
    rescaled(cache, tables, lens, 2.0 ** 120)
    got = decode(cache, tables, lens, runs, qsl, q, torch.float32, d ** -0.5)
    k, v = ref.cache_values(cache)
    want = ref.attend(q.double().numpy(), k, v, tables, lens, qsl, d ** -0.5)
    top = max(np.abs(ref.tokens_of(v, tables[s], L, 0)).max() for s, L in enumerate(lens))
    out = got.double().cpu().numpy()
    assert np.isfinite(out).all() and np.abs(out - want).max() <= REL * top
