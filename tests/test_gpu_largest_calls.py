"""The 4-bit cache and eviction at the limits that pa.h states: most query rows per KV head,
most sequences, every token protected, and queries that are not finite beside ones that
are. Tolerances are those of test_gpu_int4 and test_gpu_eviction."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import compressed as ref
from test_gpu_eviction import accumulate, check_select, filled, run_select
from test_gpu_int4 import REL, check, decode, sequences
from test_gpu_int4_range import attend_one_table, one_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("H,run,d", [(16, 255, 64), (4080, 1, 64), (15, 272, 128)])
@pytest.mark.parametrize("longest", [256, 300])       # held whole, and cut
def test_decode_of_4080_query_rows(H, run, d, longest):
    longest = max(longest, run + 1)
    lens, runs = [longest, 33, 300 if run > 1 else 1], [run, min(run, 9), min(run, 270)]
    lens = [min(n, longest) for n in lens]
    cache, tables, qsl, q = sequences(H, lens, runs, H, 1, d, torch.bfloat16)
    got = decode(cache, tables, lens, runs, qsl, q, torch.float32, d ** -0.5)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    check(got, q, cache, tables, lens, qsl, d ** -0.5, torch.float32)


@pytest.mark.parametrize("L,Hkv,d", [(100, 2, 64), (300, 1, 128)])   # held whole, and cut
def test_decode_of_8192_sequences(L, Hkv, d):
    S, H = 8192, 4
    gen = torch.Generator().manual_seed(L)
    k, v = (torch.randn((L, Hkv, d), generator=gen).half() for _ in range(2))
    q = torch.randn((S, H, d), generator=gen).half()
    cache, tables = one_table(S, L, Hkv, d, k, v)
    got = decode(cache, tables, [L] * S, [1] * S, np.arange(S + 1, dtype=np.int32), q,
                 torch.float32, d ** -0.5)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    want, _, _ = attend_one_table(cache, tables[0], L, q, d ** -0.5)
    _, values = ref.cache_values(cache)
    top = max(np.abs(ref.tokens_of(values, tables[0], L, g)).max() for g in range(Hkv))
    assert (got.double() - want).abs().max() <= REL * top


@pytest.mark.parametrize("kv", ["bf16", "int4"])
@pytest.mark.parametrize("H,run", [(4096, 1), (16, 256)])
def test_weights_of_4096_query_rows(kv, H, run):
    lens, runs, d = [300, 257], [run, max(1, run - 7)], 64
    cache, tables, src = filled(run, kv, lens, 1, d)
    q = torch.randn((sum(runs), H, d), generator=torch.Generator().manual_seed(8)).to(src)
    out, qsl = accumulate(cache, tables, lens, runs, q, d ** -0.5, None, 300)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    # 4096 weights a token are added: their sum's roundings, 2^-24 each of at most the sum
    k, _ = ref.cache_values(cache)
    w = ref.weights(q.double().numpy(), k, tables, lens, qsl, d ** -0.5, 300)
    got = out.double().cpu().numpy()
    for s, L in enumerate(lens):
        err = np.abs(got[s, :, :L] - w[s, :, :L])
        assert (err <= (6.2e-4 + 4096 * 2.0 ** -24) * w[s, :, :L] + 1e-30).all()
        assert (got[s, :, L:] == -7).all()


def test_eviction_of_65535_sequences():
    """Weights, choice and moves of one KV head of 65535 sequences of up to 20 tokens; the
    first and last thousand against the plain forms."""
    S, d, width = 65535, 64, 20
    rng = np.random.default_rng(1)
    lens = rng.integers(0, width + 1, S).astype(np.int32)
    kept = rng.integers(0, width + 1, S).astype(np.int32)
    lens[-1], kept[-1] = width, 7
    nb = 2 * S
    tables = rng.permutation(nb).astype(np.int32).reshape(S, 2)
    gen = torch.Generator(device="cuda").manual_seed(1)
    from paged_kv_cache_154_gb300.engine import PagedKVCache
    cache = PagedKVCache(nb, 1, d, "bf16")
    for t in (cache.k, cache.v):
        t.normal_(generator=gen)
    q = torch.randn((S, 2, d), generator=gen, device="cuda").bfloat16()
    bt, cl, nl = (torch.from_numpy(x).cuda() for x in (tables, lens, kept))
    w = torch.full((S, 1, width), -7.0, device="cuda")
    ws = torch.empty(pa.accumulate_weights_workspace_size(S, S, 2, 1, d, 1, width),
                     dtype=torch.uint8, device="cuda")
    pa.accumulate_weights(w, None, q, cache.k, bt, cl, width, 0.125, None, 1, nb, None, None, ws)
    old = [x.clone() for x in (cache.k, cache.v, w)]
    pos = torch.full((S, 1, width), -1, dtype=torch.int32, device="cuda")
    moves = torch.zeros((S, 1, width // 2, 2), dtype=torch.int32, device="cuda")
    counts = torch.zeros((S, 1), dtype=torch.int32, device="cuda")
    pa.evict_select(moves, counts, w, pos, w, pos, cl, nl, None, width, 1, 3)
    pa.move_tokens(cache.k, cache.v, bt, cl, moves, counts, width, nb)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    look = np.r_[0:1000, S - 1000:S]
    at = torch.from_numpy(look).cuda()
    rows = [x[bt[at].long(), 0].reshape(len(look), 32, d).double().cpu().numpy()
            for x in (old[0], old[1], cache.k, cache.v)]
    w0, w1, p1, mv, c, qs = (x[at].cpu().numpy() for x in (old[2], w, pos, moves, counts,
                                                          q.float()))
    for i, s in enumerate(look):
        L, n = int(lens[s]), min(int(kept[s]), int(lens[s]))
        want = ref.probabilities(qs[i][None].astype(np.float64), rows[0][i, :L], 0.125).sum((0, 1))
        assert np.allclose(w0[i, 0, :L], want, rtol=6.2e-4, atol=1e-7)
        m, sc, ps = ref.select(w0[i, 0], np.full(width, -1), L, n, L, 1, 3)
        assert c[i, 0] == len(m) and np.array_equal(mv[i, 0, :len(m)], m)
        assert np.array_equal(w1[i, 0, :L], sc) and np.array_equal(p1[i, 0, :L], ps)
        assert (w1[i, 0, L:] == -7).all() and (p1[i, 0, L:] == -1).all()
        for a, b in ((0, 2), (1, 3)):
            x = rows[a][i].copy()
            x[m[:, 1]] = x[m[:, 0]]
            assert np.array_equal(rows[b][i], x)


@pytest.mark.parametrize("sinks,recent", [(2 ** 31 - 1, 0), (0, 2 ** 31 - 1),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_every_token_protected(sinks, recent):
    rng = np.random.default_rng(2)
    w = rng.random((2, 3, 3000)).astype(np.float32)
    pos = np.full((2, 3, 3000), -1, np.int32)
    lens, kept = [3000, 1234], [1000, 0]
    got = run_select(w, pos, lens, kept, None, sinks, recent)
    check_select(got, w, pos, lens, kept, None, sinks, recent, np.full_like(w, -3),
                 np.full_like(pos, -9))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H", [8, 32])
def test_queries_that_are_not_finite_touch_no_other(bad, H):
    lens, runs = [700, 40], [1, 1]
    cache, tables, qsl, q = sequences(3, lens, runs, H, 2, 128, torch.bfloat16)
    q[0, 3, 5] = bad
    q[1, H - 1, :] = bad
    got = decode(cache, tables, lens, runs, qsl, q, torch.float32, 0.09)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    fine = torch.ones((2, H), dtype=torch.bool)
    fine[0, 3] = fine[1, H - 1] = False
    k, v = ref.cache_values(cache)
    want = ref.attend(torch.where(fine[..., None], q.double(), 0.0).numpy(), k, v, tables, lens, qsl,
                      0.09)
    top = max(np.abs(ref.tokens_of(v, tables[s], L, g)).max() for s, L in enumerate(lens)
              for g in range(2))
    err = np.abs(got.double().cpu().numpy() - want)[fine.numpy()]
    assert err.max() <= REL * top
    assert not torch.isfinite(got[1, H - 1]).any()
