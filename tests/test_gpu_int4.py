"""The 4-bit KV cache on the GPU against plain 64-bit forms: codes, scales and
zero points bit for bit, rows read back, attention of decode and verify steps.

Tolerance of the attention, derived before the first run. Products are exact
(codes minus zero points are integers, q is a 16-bit number scaled by a power
of two) and accumulate in fp32, so a logit is off by at most about (d + 4) half
ulps of sum |q k|: below 2^-16 of it for d <= 128. Inputs keep sum |q k| scale
under 40, so a weight is off by at most 40 * 2^-16 = 6.1e-4 relative in the
worst case and a few 1e-6 typically. P is rounded to fp16 once: half a step,
2^-11 relative per weight. Both act on the weighted sum of |v|: the error of an
output is at most (2^-11 + 6.2e-4) * sum p |v| <= 1.2e-3 * max |v| (plus half an
ulp of a 16-bit output)."""
import numpy as np
import pytest
import torch

import workloads as W
import paged_kv_cache_154_gb300 as pa
from gpu_harness import half_ulp
from oracle import compressed as ref
from paged_kv_cache_154_gb300.engine import PagedKVCache

pytestmark = pytest.mark.gpu
REL = 2.0 ** -11 + 6.2e-4


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def host_append(cache_shape, rows, slots):
    """Packed codes, scales and zero points of a pool after the rows went in."""
    nb, H, _, half = cache_shape
    g = half * 2 // ref.GROUP
    code = np.zeros(cache_shape, np.uint8)
    scale = np.zeros((nb, H, 16, g), np.float32)
    zp = np.zeros((nb, H, 16, g), np.int8)
    ok = slots >= 0
    c, s, z = ref.quantise_int4(rows[ok])
    b, o = slots[ok] // 16, slots[ok] % 16
    code[b, :, o], scale[b, :, o], zp[b, :, o] = c, s, z
    return code, scale, zp


def new_cache(num_blocks, H, d):
    return PagedKVCache(num_blocks, H, d, "int4")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy().reshape(-1)


def sequences(seed, lens, runs, H, Hkv, d, dtype, junk=True):
    """A filled INT4 cache of ragged sequences in scattered blocks. Every slot
    past a context, and every block of no sequence, holds junk: random codes,
    NaN, infinite and huge scales, zero points of any byte."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    need = [(L + 15) // 16 for L in lens]
    nb = sum(need) + 5
    order = rng.permutation(nb).astype(np.int32)
    cache = new_cache(nb, Hkv, d)
    if junk:
        for t in (cache.k, cache.v):
            t.copy_(torch.randint(0, 256, t.shape, generator=gen, dtype=torch.uint8))
        for t in (cache.k_scale, cache.v_scale):
            bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38])
            t.copy_(bad[torch.randint(0, 4, t.shape, generator=gen)])
        for t in (cache.k_zp, cache.v_zp):
            t.copy_(torch.randint(-128, 128, t.shape, generator=gen).to(torch.int8))
    tables = np.full((len(lens), max(1, max(need))), -1, np.int32)
    slots, at = [], 0
    for s, L in enumerate(lens):
        tables[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        t = np.arange(L)
        slots.append(tables[s, t // 16].astype(np.int64) * 16 + t % 16)
    slots = np.concatenate(slots)
    T = len(slots)
    k = torch.randn((T, Hkv, d), generator=gen).to(dtype)
    v = torch.randn((T, Hkv, d), generator=gen).to(dtype)
    dev = "cuda"
    pa.append_kv(k.to(dev), v.to(dev), cache.k, cache.v, torch.from_numpy(slots).to(dev),
                 nb, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)
    q = torch.randn((sum(runs), H, d), generator=gen).to(dtype)
    qsl = np.concatenate([[0], np.cumsum(runs)]).astype(np.int32)
    return cache, tables, qsl, q


def decode(cache, tables, lens, runs, qsl, q, out_dtype, scale, stream=None, out=None):
    dev = "cuda"
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device=dev) if out is None else out
    Hkv, d = cache.num_kv_heads, cache.head_dim
    size = pa.decode_workspace_size(len(lens), q.shape[0], q.shape[1], Hkv, d, max(runs),
                                    max(lens))
    pa.decode(out, q.to(dev), cache.k, cache.v, torch.from_numpy(tables).to(dev),
              torch.tensor(lens, dtype=torch.int32, device=dev), max(lens), scale,
              torch.from_numpy(qsl).to(dev) if max(runs) > 1 else None, max(runs),
              cache.num_blocks, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp, 0,
              pa.zeroed_workspace(size), stream)
    return out


def check(out, q, cache, tables, lens, qsl, scale, out_dtype):
    k, v = ref.cache_values(cache)
    want = ref.attend(q.double().numpy(), k, v, tables, lens, qsl, scale)
    got = out.double().cpu().numpy()
    live = np.concatenate([np.abs(ref.tokens_of(v, tables[s], L, g)).max(keepdims=True).ravel()
                           for s, L in enumerate(lens) for g in range(cache.num_kv_heads) if L])
    tol = REL * live.max() + (half_ulp(want, out_dtype) if out_dtype != torch.float32 else 0)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), f"max error {err.max():.3e}, largest |v| {live.max():.3e}"
    return float(err.max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(1, 1), (7, 3), (66, 8), (1000, 2)])
def test_append_is_the_quantiser_bit_for_bit(T, H, d, dtype):
    gen = torch.Generator().manual_seed(T * d)
    nb = T + 3
    rows = [torch.randn((T, H, d), generator=gen) for _ in range(2)]
    for x in rows:   # constant, all-positive, all-negative, tiny and wide groups
        x[0] = 0
        if T > 5:
            x[1] = x[1].abs() + 1
            x[2] = -x[2].abs() - 1
            x[3] *= 2.0 ** -13
            x[4] *= 1000
            x[5, :, ::7] = 0.5
    rows = [x.to(dtype) for x in rows]
    perm = torch.randperm(nb * 16, generator=gen)[:T].clone()
    if T > 6:
        perm[6] = -1
    cache = new_cache(nb, H, d)
    pa.append_kv(rows[0].cuda(), rows[1].cuda(), cache.k, cache.v, perm.cuda(), nb,
                 cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    for x, got in ((rows[0], (cache.k, cache.k_scale, cache.k_zp)),
                   (rows[1], (cache.v, cache.v_scale, cache.v_zp))):
        want = host_append((nb, H, 16, d // 2), x.float().numpy(), perm.numpy())
        for a, b in zip(got, want):
            assert np.array_equal(bits(a), np.ascontiguousarray(b).view(np.uint8).reshape(-1))


@pytest.mark.parametrize("kv", ["f16", "bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_gather_reads_back_what_the_cache_holds(kv, out_dtype, d):
    T, H, nb = 45, 3, 12
    gen = torch.Generator().manual_seed(9)
    src = torch.float16 if kv == "f16" else torch.bfloat16
    scales = (np.array([0.01, 0.02, 0.5]), np.array([0.03, 0.01, 1.0])) if kv == "fp8" else None
    cache = PagedKVCache(nb, H, d, kv, head_scales=scales)
    k, v = (torch.randn((T, H, d), generator=gen).to(src) for _ in range(2))
    slots = torch.randperm(nb * 16, generator=gen)[:T]
    pa.append_kv(k.cuda(), v.cuda(), cache.k, cache.v, slots.cuda(), nb, cache.k_scale,
                 cache.v_scale, cache.k_zp, cache.v_zp)
    # repeated and skipped slots; the skipped rows stay as they were
    ask = torch.cat([slots, slots[:3], torch.tensor([-1, -7])])
    out = [torch.full((len(ask), H, d), 7.5, dtype=out_dtype, device="cuda") for _ in range(2)]
    pa.gather_kv(out[0], out[1], cache.k, cache.v, ask.cuda(), nb, cache.k_scale, cache.v_scale,
                 cache.k_zp, cache.v_zp)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    for o, full in zip(out, ref.cache_values(cache)):
        a = ask.numpy()
        want = full[a // 16, :, a % 16]
        # one fp32 product, then one rounding to the output's type
        want = torch.from_numpy(want.astype(np.float32)).to(out_dtype).double().numpy()
        want[a < 0] = 7.5
        assert np.array_equal(o.double().cpu().numpy(), want)


CASES = [
    # lens, runs, H, Hkv, d, dtype: block and group borders, ragged ones, MHA / GQA / MQA,
    # 8 and 9 rows a KV head, several row chunks
    ([1, 15, 16, 17, 100, 513, 1500], [1] * 7, 32, 8, 128, torch.bfloat16),
    ([17, 33, 64, 100], [1] * 4, 8, 2, 64, torch.float16),
    ([33, 700, 64, 129], [1] * 4, 4, 4, 64, torch.bfloat16),
    ([1], [1], 1, 1, 128, torch.float16),
    ([2, 1, 900], [2, 1, 2], 12, 3, 128, torch.float16),
    ([40, 5, 600, 1030, 77], [5, 5, 2, 4, 1], 16, 2, 128, torch.bfloat16),
    ([40, 5, 600], [2, 5, 3], 21, 3, 64, torch.bfloat16),
    ([300, 1000, 77, 2600], [5, 1, 3, 4], 32, 1, 128, torch.bfloat16),
    ([65, 20011], [1, 1], 28, 4, 128, torch.float16),
    ([90, 41], [40, 41], 8, 2, 64, torch.float16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[2]}q{c[3]}kv_d{c[4]}_{max(c[0])}")
@pytest.mark.parametrize("out", ["f32", "q"])
def test_decode_matches_64_bits(case, out):
    lens, runs, H, Hkv, d, dtype = case
    out_dtype = torch.float32 if out == "f32" else dtype
    cache, tables, qsl, q = sequences(11 + len(lens), lens, runs, H, Hkv, d, dtype)
    got = decode(cache, tables, lens, runs, qsl, q, out_dtype, d ** -0.5)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    check(got, q, cache, tables, lens, qsl, d ** -0.5, out_dtype)


def test_rows_of_very_different_scales():
    """V scales that differ by 2^20 within a sequence: the running reference
    follows the largest, and the smaller tokens keep what fp16 weights can hold
    of them (errors stay relative to the largest value)."""
    lens, runs = [300, 64], [1, 2]
    cache, tables, qsl, q = sequences(31, lens, runs, 8, 2, 128, torch.bfloat16)
    live = np.concatenate([tables[s, :(L + 15) // 16] for s, L in enumerate(lens)])
    f = torch.exp2(torch.randint(-10, 11, (len(live),), generator=torch.Generator().manual_seed(1))
                   .float()).cuda()
    cache.v_scale[torch.from_numpy(live).long().cuda()] *= f[:, None, None, None]
    got = decode(cache, tables, lens, runs, qsl, q, torch.float32, 128 ** -0.5)
    check(got, q, cache, tables, lens, qsl, 128 ** -0.5, torch.float32)


def test_blocks_outside_the_pool_are_reported_not_read():
    lens, runs = [40, 20], [1, 1]
    cache, tables, qsl, q = sequences(5, lens, runs, 8, 2, 64, torch.float16)
    tables[0, 1] = cache.num_blocks
    decode(cache, tables, lens, runs, qsl, q, torch.float32, 0.1)
    torch.cuda.synchronize()
    assert pa.device_error() == pa.DEVERR_BAD_BLOCK
    out = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    far = torch.tensor([cache.num_blocks * 16], device="cuda")
    for call in (pa.gather_kv, pa.append_kv):
        call(out, out.clone(), cache.k, cache.v, far, cache.num_blocks, cache.k_scale,
             cache.v_scale, cache.k_zp, cache.v_zp)
        torch.cuda.synchronize()
        assert pa.device_error() == pa.DEVERR_BAD_SLOT


def test_copy_on_write_forks_of_an_int4_cache():
    """The engine on an INT4 cache: best-of-3 forks, each fork's first append
    copies the shared tail block with its scales and zero points."""
    wl = W.best_of_n("int4_bo3", 521, num_groups=2, n_forks=3, prompt_len=150,
                     shared_extra_max=9, private_max=40, num_heads=16, num_kv_heads=4,
                     head_dim=128, kv_dtype="bf16")
    cache = PagedKVCache(wl.num_blocks, 4, 128, "int4", free_order=wl.free_order)
    names = {}
    for ops in wl.phases:
        cache.run_phase(ops, names)
    si = cache.prepare_step(wl.step, names, wl.q, torch.float32)
    assert si.pairs is not None
    out = cache.step(si, wl.scale)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    # what every child holds, quantised row by row from the data before paging
    tables, lens = si.block_tables.cpu().numpy(), si.context_lens.tolist()
    kv, vv = ref.cache_values(cache)
    for s, (k, v) in enumerate(W.contiguous_kv(wl)):
        for full, x in ((kv, k), (vv, v)):
            want = ref.values_int4(*ref.quantise_int4(x.float().numpy()))
            for g in range(4):
                assert np.array_equal(ref.tokens_of(full, tables[s], lens[s], g), want[:, g])
    qsl = np.arange(len(lens) + 1)
    check(out, wl.q, cache, tables, lens, qsl, wl.scale, torch.float32)


def test_captured_replayed_and_on_another_stream():
    lens, runs = [200, 50, 1000], [1, 1, 1]
    cache, tables, qsl, q = sequences(23, lens, runs, 32, 8, 128, torch.bfloat16)
    dev = "cuda"
    eager = decode(cache, tables, lens, runs, qsl, q, torch.bfloat16, 0.088)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(eager)
    with torch.cuda.stream(side):
        decode(cache, tables, lens, runs, qsl, q, torch.bfloat16, 0.088, side, other)
    side.synchronize()
    assert torch.equal(eager, other)
    args = (q.to(dev), cache.k, cache.v, torch.from_numpy(tables).to(dev),
            torch.tensor(lens, dtype=torch.int32, device=dev), max(lens), 0.088, None, 1,
            cache.num_blocks, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp, 0,
            pa.zeroed_workspace(pa.decode_workspace_size(3, 3, 32, 8, 128, 1, 1000)))
    g = torch.cuda.CUDAGraph()
    other.zero_()
    with torch.cuda.graph(g):
        pa.decode(other, *args)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    assert torch.equal(eager, other)
    pa.decode_no_alloc(other.zero_(), *args[:-2])
    assert torch.equal(eager, other)
