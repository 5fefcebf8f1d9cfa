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
from test_gpu_int4 import REL, bits, decode, host_append, new_cache, sequences

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


def one_table(S, L, Hkv, d, k, v):
    """A cache that holds one context of L tokens (rows k, v [L, H_kv, d]), and the block
    tables of S sequences that all share it."""
    nb = (L + 15) // 16
    cache = new_cache(nb + 3, Hkv, d)
    table = np.random.default_rng(5).permutation(nb + 3)[:nb].astype(np.int32)
    t = np.arange(L)
    slots = torch.from_numpy(table[t // 16].astype(np.int64) * 16 + t % 16).cuda()
    pa.append_kv(k.cuda(), v.cuda(), cache.k, cache.v, slots, cache.num_blocks, cache.k_scale,
                 cache.v_scale, cache.k_zp, cache.v_zp)
    return cache, np.tile(table, (S, 1))


def attend_one_table(cache, table, L, q, scale):
    """64-bit attention of q [S, H, d] over the context that all of them share: outputs,
    sums of weight times |value|, and the largest weights [S, H]."""
    S, H, d = q.shape
    out, mag, top = (torch.empty((S, H, n), dtype=torch.float64, device="cuda")
                     for n in (d, d, 1))
    G = H // cache.num_kv_heads
    for g, (k, v) in enumerate(zip(*[[torch.from_numpy(ref.tokens_of(x, table, L, g)).cuda()
                                      for g in range(cache.num_kv_heads)]
                                     for x in ref.cache_values(cache)])):
        h = slice(g * G, g * G + G)
        p = torch.softmax(q[:, h].double().cuda().reshape(S * G, d) @ k.T * scale, -1)
        out[:, h] = (p @ v).reshape(S, G, d)
        mag[:, h] = (p @ v.abs()).reshape(S, G, d)
        top[:, h] = p.amax(-1).reshape(S, G, 1)
    return out, mag, top[..., 0]


@pytest.mark.parametrize("S,H,Hkv,d", [(1, 8, 2, 64), (200, 8, 1, 128), (130, 16, 1, 128),
                                       (200, 8, 1, 64)])
def test_weights_far_below_a_dominant_one(S, H, Hkv, d):
    """The first token takes nearly all of the weight and has the value 0, so that the
    others, each 2^-26 of it, make the output. A weight times its V scale is rounded to
    fp16: by 2^-11 of itself, or by 2^-32 of the largest weight times the power of two
    above the largest V scale, which the up to 15 steps of a value multiply. Logits are
    off by 2^-16 of sum |q k| scale, that is 18 of the first token: 2.8e-4 of a weight
    (the other tokens' sums are small)."""
    L = 20_000
    gen = torch.Generator().manual_seed(7)
    k = torch.randn((L, Hkv, d), generator=gen) * 0.25
    k[..., 0] = 0
    k[0] = 0
    k[0, :, 0] = 16
    v = torch.randn((L, Hkv, d), generator=gen) + 1
    v[0] = 0
    q = torch.randn((S, H, d), generator=gen) * 0.25
    scale = d ** -0.5
    q[..., 0] = 26 * float(np.log(2)) / (16 * scale)
    q = q.bfloat16()
    cache, tables = one_table(S, L, Hkv, d, k.bfloat16(), v.bfloat16())
    got = decode(cache, tables, [L] * S, [1] * S, np.arange(S + 1, dtype=np.int32), q,
                 torch.float32, scale)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    want, mag, top = attend_one_table(cache, tables[0], L, q, scale)
    assert (top > 0.99).all()
    # the tokens of the first one's piece alone are rounded against it; a call has at least
    # 1216 workers' shares, or as many as 1250 blocks make
    n = min(L, 16 * (-(-S * Hkv * 1250 // 1216) + 1))
    s_top = 2.0 ** np.ceil(np.log2(float(cache.v_scale[tables[0].tolist()].max())))
    tol = mag * (2.0 ** -11 + 5.6e-4) + n * 15 * s_top * 2.0 ** -32
    err = (got.double() - want).abs()
    assert (err <= tol).all(), ((err - tol).max(), want.abs().max())


@pytest.mark.parametrize("H,d", [(16, 128), (32, 128), (8, 64), (32, 64)])
def test_small_averages_over_long_shares(H, d):
    """Nearly even weights over shares of several hundred blocks: values of either sign
    average to a hundredth of them, where what the accumulation loses would show. The
    bound is that of test_small_averages_of_long_contexts: 2^-11 / sqrt(3) of the norm in
    the mean square for the fp16 weights, up to 2^-11 with the accumulation, for the
    elements of the low and of the high halves of bytes."""
    S, L, Hkv = 256, 32768, 2          # 1048576 blocks over at most 1824 workers
    gen = torch.Generator().manual_seed(d + H)
    k, v = (torch.randn((L, Hkv, d), generator=gen).bfloat16() for _ in range(2))
    q = torch.randn((S, H, d), generator=gen).bfloat16()
    scale = 0.25 * d ** -0.5
    cache, tables = one_table(S, L, Hkv, d, k, v)
    got = decode(cache, tables, [L] * S, [1] * S, np.arange(S + 1, dtype=np.int32), q,
                 torch.float32, scale)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    want, mag, _ = attend_one_table(cache, tables[0], L, q, scale)
    err = got.double() - want
    for half in (0, 1):
        e, w = err[..., half::2].norm(), want[..., half::2].norm()
        print(f"half {half}: {e / w:.2e} of the norm, which is {w / mag[..., half::2].norm():.1e}")
        assert e <= 2.0 ** -11 * w


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", ["mixed", "positive", "negative"])
def test_append_at_the_ends_of_fp32_is_the_quantiser(d, sign):
    """Groups whose range is subnormal, next to 1e-28 and 1e30 (where the append changes
    its way of dividing) or near the largest that is finite: codes, scales and zero points
    bit for bit, and read back at their values."""
    factors = torch.tensor([1e-40, 1e-39, 1e-38, 1e-37, 1e-31, 1e-29, 1.7e-29, 2e-29, 2.3e-29,
                            2.7e-29, 3e-29, 1e-28, 1e-20, 1e29, 1.7e29, 2e29, 2.3e29, 2.7e29,
                            3e29, 1e30, 1e31, 1e33, 1e36, 3e37], dtype=torch.float64)
    T, H = 40 * len(factors), 3
    gen = torch.Generator().manual_seed(d)
    rows = []
    for _ in range(2):
        x = torch.randn((T, H, d), generator=gen, dtype=torch.float64).clamp(-4.5, 4.5)
        x = {"mixed": x, "positive": x.abs(), "negative": -x.abs()}[sign]
        x[::7, :, ::5] = 0
        rows.append((x * factors[torch.randint(len(factors), (T, 1, 1), generator=gen)]).bfloat16())
    nb = T // 16 + 4
    slots = torch.randperm(nb * 16, generator=gen)[:T]
    cache = new_cache(nb, H, d)
    on = (cache.k, cache.v, slots.cuda(), nb, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)
    pa.append_kv(rows[0].cuda(), rows[1].cuda(), *on)
    back = {t: [torch.empty((T, H, d), dtype=t, device="cuda") for _ in range(2)]
            for t in (torch.float32, torch.bfloat16)}
    for out in back.values():
        pa.gather_kv(*out, *on)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    both = []
    for i, (x, got) in enumerate(((rows[0], (cache.k, cache.k_scale, cache.k_zp)),
                                  (rows[1], (cache.v, cache.v_scale, cache.v_zp)))):
        f = x.float().numpy()
        assert np.isfinite(f).all()
        span = (np.maximum(f.reshape(T, H, -1, 64).max(-1), 0) -
                np.minimum(f.reshape(T, H, -1, 64).min(-1), 0))
        assert np.isfinite(span).all()
        both += [((span > lo) & (span < hi)).any() for lo, hi in
                 ((0, 1e-37), (5e-29, 1e-28), (1e-28, 2e-28), (5e29, 1e30), (1e30, 2e30), (1e37, 3e38))]
        want = host_append((nb, H, 16, d // 2), f, slots.numpy())
        for a, b in zip(got, want):
            assert np.array_equal(bits(a), np.ascontiguousarray(b).view(np.uint8).reshape(-1))
        held = ref.values_int4(*ref.quantise_int4(f))
        assert np.array_equal(back[torch.float32][i].cpu().numpy(), held.astype(np.float32))
        assert torch.equal(back[torch.bfloat16][i].cpu(),
                           torch.from_numpy(held.astype(np.float32)).bfloat16())
    assert all(both)                          # every side of both thresholds is met


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_group_that_is_not_finite_touches_no_other(bad):
    T, H, d, nb = 50, 3, 128, 8
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((T, H, d), generator=gen).bfloat16()
    y = x.clone()
    y[7, 1, 70] = bad
    y[9, 2, 3] = bad
    slots = torch.randperm(nb * 16, generator=gen)[:T]
    caches = []
    for rows in (x, y):
        c = new_cache(nb, H, d)
        pa.append_kv(rows.cuda(), rows.cuda(), c.k, c.v, slots.cuda(), nb, c.k_scale, c.v_scale,
                     c.k_zp, c.v_zp)
        caches.append([a.reshape(nb, H, 16, 2, -1)[slots.cuda() // 16, :, slots.cuda() % 16]
                       .cpu().contiguous().view(torch.uint8) for a in c.arrays()])
    keep = torch.ones((T, H, 2), dtype=torch.bool)
    keep[7, 1, 1] = keep[9, 2, 0] = False
    for a, b in zip(*caches):
        assert torch.equal(a[keep], b[keep])
