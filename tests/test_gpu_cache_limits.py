"""The 4-bit cache and eviction at their limits: lengths around the one at which
decode starts to cut contexts, padded batches, caches past 4 GB, selections of
every cluster and block size, captured runs that share a workspace, and the
checks of PA_VALIDATE. Tolerances are those of test_gpu_int4 and
test_gpu_eviction; comparisons of two runs of one kernel are bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import compressed as ref
from paged_kv_cache_154_gb300.engine import PagedKVCache
from test_gpu_eviction import accumulate, check as check_weights
from test_gpu_eviction import check_select, filled, run_select
from test_gpu_int4 import check, decode, sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("lens,runs,H,Hkv,d", [
    ([255, 256, 1], [1, 1, 1], 8, 2, 128),       # contexts held whole
    ([257, 256, 1], [1, 1, 1], 8, 2, 128),       # cut
    ([256, 250, 40], [40, 1, 3], 8, 4, 64),      # whole, several chunks of rows
    ([272, 250, 40], [40, 1, 3], 8, 4, 64),
    ([256, 30], [17, 30], 24, 2, 128),
])
def test_lengths_around_the_uncut_limit(lens, runs, H, Hkv, d):
    cache, tables, qsl, q = sequences(max(lens), lens, runs, H, Hkv, d, torch.bfloat16)
    got = decode(cache, tables, lens, runs, qsl, q, torch.float32, d ** -0.5)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    check(got, q, cache, tables, lens, qsl, d ** -0.5, torch.float32)


@pytest.mark.parametrize("lens,runs,H,Hkv,d", [
    ([257 + 7 * i % 90 for i in range(250)], [1] * 250, 16, 8, 64),      # more segments than workers
    ([260 + 11 * i % 60 for i in range(70)], [5, 1] * 35, 64, 8, 128),   # and of two row chunks
    ([300, 40000, 1], [1, 1, 1], 8, 2, 128),                             # hundreds of pieces
    ([3000, 25, 17], [40, 2, 3], 8, 2, 64),
])
def test_cut_segments_merge_inside_their_workspace(lens, runs, H, Hkv, d):
    """However a call is cut: right answers, and nothing written past the workspace
    and the output, whatever the workspace held before."""
    cache, tables, qsl, q = sequences(len(lens), lens, runs, H, Hkv, d, torch.bfloat16, junk=False)
    size = pa.decode_workspace_size(len(lens), q.shape[0], H, Hkv, d, max(runs), max(lens))
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:pa.ARRIVAL_BYTES] = 0
    out = torch.full((q.shape[0] + 8, H, d), 7.0, device="cuda")
    pa.decode(out[:q.shape[0]], q.cuda(), cache.k, cache.v, torch.from_numpy(tables).cuda(),
              torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens), d ** -0.5,
              torch.from_numpy(qsl).cuda() if max(runs) > 1 else None, max(runs),
              cache.num_blocks, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp, 0, ws[:size])
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    assert (ws[size:] == 0xA5).all() and (out[q.shape[0]:] == 7).all()
    assert (ws[:pa.ARRIVAL_BYTES] == 0).all()
    check(out[:q.shape[0]], q, cache, tables, lens, qsl, d ** -0.5, torch.float32)


@pytest.mark.parametrize("d", [64, 128])
def test_small_averages_of_long_contexts(d):
    """Nearly even weights over a long context average values of either sign to
    a hundredth of them, where errors of the accumulation would show. Weights are
    rounded to fp16, off by at most 2^-11 and 2^-11 / sqrt(3) in the mean square;
    the same weights make the output, so its error is that share of its norm,
    for the elements of the low halves of bytes and for those of the high ones.
    The rest of 2^-11 is left to the accumulation."""
    lens, runs = [60_000], [1]
    cache, tables, qsl, q = sequences(d, lens, runs, 16, 2, d, torch.bfloat16)
    got = decode(cache, tables, lens, runs, qsl, q, torch.float32, 0.25 * d ** -0.5)
    k, v = ref.cache_values(cache)
    want = ref.attend(q.double().numpy(), k, v, tables, lens, qsl, 0.25 * d ** -0.5)
    err = got.double().cpu().numpy() - want
    for half in (0, 1):
        e, w = err[..., half::2], want[..., half::2]
        assert np.linalg.norm(e) <= 2.0 ** -11 * np.linalg.norm(w)


@pytest.mark.parametrize("long", [100, 900])
def test_rows_of_empty_sequences_are_left_as_they_were(long):
    lens, runs = [0, long, 0, 33, 0], [1] * 5
    cache, tables, qsl, q = sequences(3, lens, runs, 8, 2, 128, torch.float16)
    out = torch.full(q.shape, 5.5, device="cuda")
    decode(cache, tables, lens, runs, qsl, q, torch.float32, 0.09, out=out)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    live = [1, 3]
    assert (out[[0, 2, 4]] == 5.5).all()
    check(out[live], q[live], cache, tables[live], [long, 33], np.arange(3), 0.09, torch.float32)


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("longest", [4096, 4097])     # 16 tiles of many rows, and one more
def test_weights_of_many_rows_and_tiles(kv, longest):
    lens, runs, H, Hkv, d = [longest, 300, 0, 31], [21, 40, 0, 1], 8, 2, 64 if kv == "fp8" else 128
    cache, tables, src = filled(longest, kv, lens, Hkv, d)
    q = torch.randn((sum(runs), H, d), generator=torch.Generator().manual_seed(3)).to(src)
    before = torch.rand((4, Hkv, longest), device="cuda")
    out, qsl = accumulate(cache, tables, lens, runs, q, d ** -0.5, before, longest)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    check_weights(out, cache, tables, lens, qsl, q, d ** -0.5, before, longest)


# num_blocks whose K alone passes 4 GB: 16 tokens x 8 heads x 128 elements a block
@pytest.mark.parametrize("kv,num_blocks", [("int4", 560_000), ("bf16", 140_000)])
def test_caches_past_4_gb(kv, num_blocks):
    lens, H, d = [700, 33], 8, 128
    small, tables, src = filled(4, kv, lens, H, d)
    far = num_blocks - small.num_blocks
    big = PagedKVCache(num_blocks, H, d, kv)
    for a, b in zip(big.arrays(), small.arrays()):
        a[far:] = b
    far_tables = np.where(tables >= 0, tables + far, -1).astype(np.int32)
    gen = torch.Generator().manual_seed(1)
    q = torch.randn((2, 32, d), generator=gen).to(src)
    qsl = np.arange(3, dtype=np.int32)

    def same():
        torch.cuda.synchronize()
        assert pa.device_error() == 0
        for a, b in zip(big.arrays(), small.arrays()):
            assert torch.equal(a[far:].reshape(-1).view(torch.uint8),
                               b.reshape(-1).view(torch.uint8))

    def both(call):
        return [call(c, t) for c, t in ((small, tables), (big, far_tables))]

    def on(cache):
        return (cache.num_blocks, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)

    a, b = both(lambda c, t: decode(c, t, lens, [1, 1], qsl, q, torch.float32, 0.09))
    assert torch.equal(a, b)
    a, b = both(lambda c, t: accumulate(c, t, lens, [1, 1], q, 0.09, None, 700)[0])
    assert torch.equal(a, b)
    run = torch.randn((40, 32, d), generator=gen).to(src)
    a, b = both(lambda c, t: accumulate(c, t, lens, [30, 10], run, 0.09, None, 700)[0])
    assert torch.equal(a, b)
    rows = [torch.randn((3, H, d), generator=gen).to(src).cuda() for _ in range(2)]
    at = torch.tensor([5, 16 * 20 + 3, 16 * small.num_blocks - 1])

    def append(c, t):
        slots = (at + 16 * (c.num_blocks - small.num_blocks)).cuda()
        pa.append_kv(*rows, c.k, c.v, slots, *on(c))
        out = [torch.empty_like(r) for r in rows]
        pa.gather_kv(*out, c.k, c.v, slots, *on(c))
        return torch.stack(out)
    a, b = both(append)
    assert torch.equal(a, b)
    same()
    moves = torch.zeros((2, H, 350, 2), dtype=torch.int32, device="cuda")
    moves[0, :, :300, 0] = torch.arange(400, 700)
    moves[0, :, :300, 1] = torch.randperm(300, generator=gen).int()
    counts = torch.tensor([[300] * H, [0] * H], dtype=torch.int32, device="cuda")
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def move(c, t):
        pa.move_tokens(c.k, c.v, torch.from_numpy(t).cuda(), cl, moves, counts, 700, *on(c))
        p = torch.tensor([[0, 2], [1, 3]], dtype=torch.int32, device="cuda")
        pa.copy_blocks(c.k, c.v, p + (c.num_blocks - small.num_blocks), *on(c))
    both(move)
    same()


# sequences x heads, tokens: every number of CTAs a row (1, 2, 4, 8) and threads a CTA
@pytest.mark.parametrize("S,H,L", [
    (20, 8, 1200), (20, 8, 3001), (20, 8, 6000),     # 1 CTA a row
    (10, 8, 2500), (10, 8, 5003), (10, 8, 10000),    # 2
    (5, 8, 4800), (5, 8, 10001), (5, 8, 20000),      # 4
    (1, 2, 9000), (1, 2, 30001), (1, 2, 70000),      # 8
    (1, 1, 362_000),                                 # keys that do not fit shared memory
])
@pytest.mark.parametrize("in_place", [False, True])
def test_selection_of_every_split(S, H, L, in_place):
    rng = np.random.default_rng(L)
    w = np.floor(np.exp(3 * rng.standard_normal((S, H, L)))).astype(np.float32) / 8
    lens = [L] + [int(x) for x in rng.integers(0, L + 1, S - 1)]
    kept = [L // 3] + [int(x) for x in rng.integers(0, L, S - 1)]
    pos = np.full((S, H, L), -1, np.int32)
    pos[:, :, :500] = rng.permutation(500)
    got = run_select(w, pos, lens, kept, None, 4, 100, in_place)
    past = (w, pos) if in_place else (np.full_like(w, -3), np.full_like(pos, -9))
    check_select(got, w, pos, lens, kept, None, 4, 100, *past)


def test_a_captured_eviction_replays_to_what_eager_calls_do():
    """accumulate, select and move in one graph, over a second graph's workspace;
    each replay starts from the same cache and scores."""
    lens, H, d, W = [600, 90], 2, 64, 600
    cache, tables, src = filled(8, "int4", lens, H, d)
    gen = torch.Generator().manual_seed(2)
    q = torch.randn((2, 8, d), generator=gen).to(src).cuda()
    bt, cl = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    kept = torch.tensor([200, 90], dtype=torch.int32).cuda()
    scores = torch.empty((2, H, W), device="cuda")
    pos = torch.empty((2, H, W), dtype=torch.int32, device="cuda")
    moves = torch.empty((2, H, 300, 2), dtype=torch.int32, device="cuda")
    counts = torch.empty((2, H), dtype=torch.int32, device="cuda")
    out = torch.empty((2, 8, d), dtype=src, device="cuda")
    start = [a.clone() for a in cache.arrays()]
    ws = torch.empty(pa.accumulate_weights_workspace_size(2, 2, 8, H, d, 1, 600),
                     dtype=torch.uint8, device="cuda")
    dws = pa.zeroed_workspace(pa.decode_workspace_size(2, 2, 8, H, d, 1, 600))
    scales = (cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)

    def reset():
        for a, b in zip(cache.arrays(), start):
            a.copy_(b)
        scores.zero_()
        pos.fill_(-1)

    def evict():
        pa.accumulate_weights(scores, scores, q, cache.k, bt, cl, 600, 0.1, None, 1,
                              cache.num_blocks, cache.k_scale, cache.k_zp, ws)
        pa.evict_select(moves, counts, scores, pos, scores, pos, cl, kept, None, 600, 2, 8)
        pa.move_tokens(cache.k, cache.v, bt, cl, moves, counts, 600, cache.num_blocks, *scales)

    def attend():
        pa.decode(out, q, cache.k, cache.v, bt, kept, 200, 0.1, None, 1, cache.num_blocks,
                  *scales, 0, dws)
        pa.accumulate_weights(scores, scores, q, cache.k, bt, kept, 600, 0.1, None, 1,
                              cache.num_blocks, cache.k_scale, cache.k_zp, ws)

    reset()
    evict()
    attend()
    want = [a.clone() for a in (*cache.arrays(), scores, pos, counts, out)]
    graphs = []
    for fn in (evict, attend):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        graphs.append(g)
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side, torch.cuda.current_stream()):
        with torch.cuda.stream(stream):
            reset()
            out.zero_()
            for g in graphs:
                g.replay()
        stream.synchronize()
        assert pa.device_error() == 0
        for a, b in zip((*cache.arrays(), scores, pos, counts, out), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_validation_names_what_is_wrong(monkeypatch):
    monkeypatch.setenv("PA_VALIDATE", "1")
    lens, H, d = [40, 20], 2, 64
    cache, tables, src = filled(9, "int4", lens, H, d)
    scales = (cache.num_blocks, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)
    rows = torch.zeros((1, H, d), dtype=src, device="cuda")
    far = torch.tensor([cache.num_blocks * 16], device="cuda")
    for call in (pa.append_kv, pa.gather_kv):
        with pytest.raises(pa.PAError, match="outside the pool"):
            call(rows, rows.clone(), cache.k, cache.v, far, *scales)
    q = torch.zeros((2, 4, d), dtype=src)
    bad = tables.copy()
    bad[0, 1] = cache.num_blocks
    with pytest.raises(pa.PAError):
        accumulate(cache, bad, lens, [1, 1], q, 0.1, None, 40)
    with pytest.raises(pa.PAError, match="context_len"):
        accumulate(cache, tables, lens, [1, 1], q, 0.1, None, 40, max_len=30)
    with pytest.raises(pa.PAError, match="context_len"):
        run_select(np.zeros((1, 1, 10), np.float32), None, [-1], [3], None, 0, 0)
    with pytest.raises(pa.PAError, match="total_len"):
        run_select(np.zeros((1, 1, 10), np.float32), None, [9], [3], [8], 0, 0)
    bt, cl = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for pairs, text in (([[40, 0]], "outside"), ([[30, 1], [31, 1]], "twice"),
                        ([[30, 1], [1, 2]], "twice"), ([[0, 0]] * 21, "at most")):
        moves = torch.zeros((2, H, 20, 2), dtype=torch.int32, device="cuda")
        n = min(20, len(pairs))
        moves[0, 1, :n] = torch.tensor(pairs[:n], dtype=torch.int32)
        counts = torch.tensor([[0, len(pairs)], [0, 0]], dtype=torch.int32, device="cuda")
        with pytest.raises(pa.PAError, match=text):
            pa.move_tokens(cache.k, cache.v, bt, cl, moves, counts, 40, *scales)
    # and what is right passes
    out, _ = accumulate(cache, tables, lens, [1, 1], q, 0.1, None, 40)
    assert torch.allclose(out[0, :, :40], torch.full((2, 40), 2 / 40, device="cuda"), rtol=1e-5)
    moves[0, 1, 0] = torch.tensor([30, 1], dtype=torch.int32)
    counts[0, 1] = 1
    pa.move_tokens(cache.k, cache.v, bt, cl, moves, counts, 40, *scales)


def test_arguments_of_a_wrong_type_are_refused():
    cache, tables, src = filled(10, "bf16", [40], 1, 64)
    cl, bt = torch.tensor([40], device="cuda"), torch.from_numpy(tables).cuda()   # int64 lengths
    w, pos = torch.zeros((1, 1, 40), device="cuda"), torch.zeros((1, 1, 40), dtype=torch.int32).cuda()
    moves, counts = pos.new_zeros((1, 1, 20, 2)), pos.new_zeros((1, 1))
    with pytest.raises(ValueError, match="context_lens"):
        pa.evict_select(moves, counts, w, pos, w, pos, cl, cl.int(), None, 40)
    with pytest.raises(ValueError, match="new_lens"):
        pa.evict_select(moves, counts, w, pos, w, pos, cl.int(), cl, None, 40)
    with pytest.raises(ValueError, match="context_lens"):
        pa.move_tokens(cache.k, cache.v, bt, cl, moves, counts, 40)
    with pytest.raises(ValueError, match="block_tables"):
        pa.accumulate_weights(w, None, torch.zeros((1, 1, 64), dtype=src).cuda(), cache.k,
                              bt.long(), cl.int(), 40, 0.1)
