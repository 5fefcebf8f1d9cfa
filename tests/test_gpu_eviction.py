"""Accumulated attention weights and eviction on the GPU against plain 64-bit
forms.

Tolerance of a weight, derived before the first run: logits are sums of exact
products in fp32 (see the decode tests), off by at most 2^-16 of sum |q k|; the
inputs keep sum |q k| scale under 40 (normal rows, d <= 128), so a weight is off
by at most 40 * 2^-16 = 6.1e-4 relative, plus 2^-20 for the exponential, the
sums and the division. An output adds `rows` such weights to its input: error
<= 6.2e-4 * (its own sum of weights) + 2^-23 * |output|."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import compressed as ref
from paged_kv_cache_154_gb300.engine import PagedKVCache

pytestmark = pytest.mark.gpu
REL = 6.2e-4


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def filled(seed, kv, lens, Hkv, d, extra=5):
    """A cache of ragged sequences in scattered blocks; slots past a context and
    spare blocks hold NaN (16-bit, scales) or any code."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    need = [(L + 15) // 16 for L in lens]
    nb = sum(need) + extra
    order = rng.permutation(nb).astype(np.int32)
    heads = (np.full(Hkv, 0.01), np.full(Hkv, 0.02)) if kv == "fp8" else None
    cache = PagedKVCache(nb, Hkv, d, kv, head_scales=heads)
    for t in cache.arrays():
        if t.is_floating_point() and kv != "fp8":
            t.fill_(float("nan"))
        elif kv == "fp8":
            t.view(torch.uint8).fill_(0x7F)          # NaN
        else:
            t.copy_(torch.randint(0, 100, t.shape, generator=gen).to(t.dtype))
    tables = np.full((len(lens), max(1, max(need))), -1, np.int32)
    slots, at = [], 0
    for s, L in enumerate(lens):
        tables[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        t = np.arange(L)
        slots.append(tables[s, t // 16].astype(np.int64) * 16 + t % 16)
    slots = np.concatenate(slots)
    src = torch.float16 if kv == "f16" else torch.bfloat16
    k, v = (torch.randn((len(slots), Hkv, d), generator=gen).to(src) for _ in range(2))
    pa.append_kv(k.cuda(), v.cuda(), cache.k, cache.v, torch.from_numpy(slots).cuda(), nb,
                 cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)
    return cache, tables, src


def accumulate(cache, tables, lens, runs, q, scale, before, width, max_len=None, out=None):
    S, H = len(lens), cache.num_kv_heads
    qsl = np.concatenate([[0], np.cumsum(runs)]).astype(np.int32)
    max_len = max(1, max(lens)) if max_len is None else max_len
    max_run = max(1, max(runs))
    out = torch.full((S, H, width), -7.0, device="cuda") if out is None else out
    ws = torch.empty(pa.accumulate_weights_workspace_size(S, q.shape[0], q.shape[1], H,
                                                          cache.head_dim, max_run, max_len),
                     dtype=torch.uint8, device="cuda").fill_(0xFF)   # NaN where not written
    pa.accumulate_weights(out, before, q.cuda(), cache.k, torch.from_numpy(tables).cuda(),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len, scale,
                          None if runs == [1] * S else torch.from_numpy(qsl).cuda(), max_run,
                          cache.num_blocks, cache.k_scale, cache.k_zp, ws)
    return out, qsl


def check(out, cache, tables, lens, qsl, q, scale, before, width):
    k, _ = ref.cache_values(cache)
    w = ref.weights(q.double().numpy(), k, tables, lens, qsl, scale, width)
    start = np.zeros_like(w) if before is None else before.double().cpu().numpy()
    got = out.double().cpu().numpy()
    for s, L in enumerate(lens):
        want = start[s, :, :L] + w[s, :, :L]
        err = np.abs(got[s, :, :L] - want)
        assert (err <= REL * w[s, :, :L] + 2.0 ** -23 * np.abs(want) + 1e-30).all(), err.max()
        assert (got[s, :, L:] == -7).all()


CASES = [
    # lens, runs, H, Hkv, d: 1 to 16 rows a KV head (stored logits), and more (computed again)
    ([1, 15, 16, 17, 100, 511, 512, 513], [1] * 8, 8, 2, 128),
    ([33, 2000], [1, 1], 3, 3, 64),
    ([40, 5, 700], [2, 5, 1], 12, 6, 64),
    ([300, 90], [2, 4], 28, 4, 128),
    ([700, 0, 65, 1], [3, 0, 4, 1], 16, 1, 128),
    ([1500, 129, 40], [32, 17, 40], 8, 2, 64),
    ([260, 530], [5, 9], 14, 2, 128),
    ([5, 9], [7, 3], 2, 1, 64),          # a run longer than its context: rows that see nothing
]


@pytest.mark.parametrize("kv", ["f16", "bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[2]}q{c[3]}kv_d{c[4]}_run{max(c[1])}")
def test_weights_match_64_bits(case, kv):
    lens, runs, H, Hkv, d = case
    cache, tables, src = filled(3 + len(lens), kv, lens, Hkv, d)
    q = torch.randn((sum(runs), H, d), generator=torch.Generator().manual_seed(8)).to(src)
    width = max(lens) + 3
    before = torch.rand((len(lens), Hkv, width), device="cuda")
    for b in (before, None):
        out, qsl = accumulate(cache, tables, lens, runs, q, d ** -0.5, b, width)
        torch.cuda.synchronize()
        assert pa.device_error() == 0
        check(out, cache, tables, lens, qsl, q, d ** -0.5, b, width)


def test_many_sequences_too_long_to_store_are_computed_again():
    """A padded batch whose stored logits would pass the buffer's limit: the
    same weights, from logits computed twice, with a graph's largest length."""
    lens, runs, H, Hkv, d = [700, 20, 1], [1, 1, 1], 16, 1, 64
    cache, tables, src = filled(4, "bf16", lens, Hkv, d)
    q = torch.randn((3, H, d), generator=torch.Generator().manual_seed(8)).to(src)
    far = 1 << 21                        # 3 x 2 M tokens x 16 rows x 4 bytes: 400 MB
    wide = np.full((3, far // 16), -1, np.int32)
    wide[:, :tables.shape[1]] = tables
    few, qsl = accumulate(cache, tables, lens, runs, q, 0.125, None, 800)
    size = [pa.accumulate_weights_workspace_size(3, 3, H, Hkv, d, 1, n) for n in (800, far)]
    assert size[1] < 16 << 20
    out = torch.full((3, Hkv, far), -7.0, device="cuda")
    accumulate(cache, wide, lens, runs, q, 0.125, None, far, far, out)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    check(out[..., :800], cache, tables, lens, qsl, q, 0.125, None, 800)
    check(few, cache, tables, lens, qsl, q, 0.125, None, 800)
    assert (out[..., 800:] == -7).all()


def test_weights_in_place_on_a_stream_and_replayed():
    lens, runs, H, Hkv, d = [900, 33], [1, 1], 8, 2, 128
    cache, tables, src = filled(6, "int4", lens, Hkv, d)
    q = torch.randn((2, H, d), generator=torch.Generator().manual_seed(8)).to(src)
    first, qsl = accumulate(cache, tables, lens, runs, q, 0.09, None, 900)
    both = torch.zeros_like(first)
    ws = torch.empty(pa.accumulate_weights_workspace_size(2, 2, H, Hkv, d, 1, 900),
                     dtype=torch.uint8, device="cuda")
    args = (q.cuda(), cache.k, torch.from_numpy(tables).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), 900, 0.09, None, 1,
            cache.num_blocks, cache.k_scale, cache.k_zp, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.accumulate_weights(both, both, *args)
    for _ in range(2):
        g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.accumulate_weights(both, both, *args, stream=side)
    side.synchronize()
    a, b = first[0].double(), both[0].double()
    assert torch.allclose(b, 3 * a, rtol=2.0 ** -22, atol=0)
    # every row's weights sum to the number of its query heads per KV head
    assert torch.allclose(first[0].double().sum(-1), torch.full((2,), 4.0, device="cuda").double(),
                          rtol=1e-5)


def test_weights_of_a_block_outside_the_pool_are_reported():
    cache, tables, src = filled(7, "bf16", [40], 1, 64)
    q = torch.randn((1, 4, 64)).to(src)
    tables[0, 1] = cache.num_blocks + 3
    accumulate(cache, tables, [40], [1], q, 0.1, None, 40)
    torch.cuda.synchronize()
    assert pa.device_error() == pa.DEVERR_BAD_BLOCK


# ---------------------------------------------------------------------------
# selection and moves
# ---------------------------------------------------------------------------

def run_select(scores, positions, lens, kept, total, sinks, recent, in_place=False):
    S, H, W = scores.shape
    dev = "cuda"
    ints = [None if a is None else torch.tensor(a, dtype=torch.int32, device=dev)
            for a in (lens, kept, total)]
    w = torch.from_numpy(scores).to(dev)
    pos = None if positions is None else torch.from_numpy(positions).to(dev)
    w_out = w if in_place else torch.full_like(w, -3)
    p_out = pos if in_place else torch.full((S, H, W), -9, dtype=torch.int32, device=dev)
    max_len = max(1, max(lens))
    moves = torch.full((S, H, max(1, max_len // 2), 2), -5, dtype=torch.int32, device=dev)
    counts = torch.full((S, H), -5, dtype=torch.int32, device=dev)
    pa.evict_select(moves, counts, w_out, p_out, w, pos, *ints, max_len, sinks, recent)
    torch.cuda.synchronize()
    return moves.cpu().numpy(), counts.cpu().numpy(), w_out.cpu().numpy(), p_out.cpu().numpy()


def check_select(got, scores, positions, lens, kept, total, sinks, recent, w_past, p_past):
    moves, counts, w_out, p_out = got
    S, H, W = scores.shape
    for s in range(S):
        L = lens[s]
        for g in range(H):
            pos = np.full(W, -1) if positions is None else positions[s, g]
            mv, w, p = ref.select(scores[s, g], pos, L, kept[s], L if total is None else total[s],
                                  sinks, recent)
            assert counts[s, g] == len(mv)
            assert np.array_equal(moves[s, g, :len(mv)], mv)
            assert (moves[s, g, len(mv):] == -5).all()
            assert np.array_equal(w_out[s, g, :L], w, equal_nan=True)
            assert np.array_equal(p_out[s, g, :L], p)
            assert np.array_equal(w_out[s, g, L:], w_past[s, g, L:], equal_nan=True)
            assert np.array_equal(p_out[s, g, L:], p_past[s, g, L:])


LENGTHS = [
    # lens, kept: nothing, all, one, block borders, more than there are, a negative budget
    ([1, 1, 2, 17, 100], [0, 1, 1, 16, 40]),
    ([64, 64, 64, 0], [0, 64, 70, 5]),
    ([513, 1000, 37], [-1, 999, 1]),
    ([5000, 4097], [1024, 2048]),
    ([40000], [9000]),
]


@pytest.mark.parametrize("lens,kept", LENGTHS)
@pytest.mark.parametrize("kind", ["smooth", "ties", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
def test_selection_is_exact(lens, kept, kind, in_place):
    rng = np.random.default_rng(len(lens) + lens[0])
    S, H, W = len(lens), 3, max(lens) + 5
    w = np.exp(2 * rng.standard_normal((S, H, W))).astype(np.float32)
    if kind == "ties":
        w = np.floor(w).astype(np.float32)       # most scores are 0 or 1
    if kind == "odd":
        w[rng.random(w.shape) < 0.2] = 0
        w[rng.random(w.shape) < 0.1] = -0.0
        w[rng.random(w.shape) < 0.1] = np.nan
        w[rng.random(w.shape) < 0.05] = np.inf
        w[rng.random(w.shape) < 0.05] = -np.inf
        w[rng.random(w.shape) < 0.1] *= -1
        w[rng.random(w.shape) < 0.05] = 1e-42    # subnormal
    total = [L + 6 * (s + 1) for s, L in enumerate(lens)]
    pos = np.full((S, H, W), -1, np.int32)
    for s, L in enumerate(lens):                 # some slots filled by an earlier eviction
        n = min(L // 2, 200)
        for g in range(H):
            pos[s, g, :n] = rng.permutation(n + 6 * (s + 1))[:n]
    for sinks, recent in ((0, 0), (4, 16), (3, 100000)):
        got = run_select(w, pos, lens, kept, total, sinks, recent, in_place)
        past = (w, pos) if in_place else (np.full_like(w, -3), np.full_like(pos, -9))
        check_select(got, w, pos, lens, kept, total, sinks, recent, *past)


def test_selection_without_positions_or_totals():
    rng = np.random.default_rng(2)
    w = rng.random((2, 2, 300)).astype(np.float32)
    got = run_select(w, None, [300, 200], [100, 50], None, 2, 8)
    check_select(got, w, None, [300, 200], [100, 50], None, 2, 8, np.full_like(w, -3),
                 np.full(w.shape, -9))


@pytest.mark.parametrize("kv", ["f16", "bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("d", [64, 128])
def test_moves_carry_rows_scales_and_zero_points(kv, d):
    lens, H = [100, 33, 700, 1, 0], 3
    cache, tables, _ = filled(12, kv, lens, H, d)
    rng = np.random.default_rng(1)
    S, most = len(lens), 350
    moves = np.full((S, H, most, 2), 1 << 30, np.int32)     # entries past the count: not read
    counts = np.zeros((S, H), np.int32)
    want = [a.clone() for a in cache.arrays()]
    for s, L in enumerate(lens):
        for g in range(H):
            n = int(rng.integers(0, L // 2 + 1))
            slots = rng.permutation(L)[:2 * n].reshape(2, n)
            counts[s, g] = n
            moves[s, g, :n] = slots.T
            for a in want:
                for i, j in slots.T:
                    a[tables[s, j // 16], g, j % 16] = a[tables[s, i // 16], g, i % 16].clone()
    pa.move_tokens(cache.k, cache.v, torch.from_numpy(tables).cuda(),
                   torch.tensor(lens, dtype=torch.int32, device="cuda"),
                   torch.from_numpy(moves).cuda(), torch.from_numpy(counts).cuda(), max(lens),
                   cache.num_blocks, cache.k_scale, cache.v_scale, cache.k_zp, cache.v_zp)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    for a, b in zip(cache.arrays(), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_bad_moves_are_reported_and_skipped():
    cache, tables, _ = filled(13, "bf16", [40, 40], 1, 64)
    before = [a.clone() for a in cache.arrays()]
    lens = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    bt = torch.from_numpy(tables).cuda()
    for bad in ([40, 0], [0, 40], [-1, 0], [0, -5]):
        moves = torch.zeros((2, 1, 20, 2), dtype=torch.int32, device="cuda")
        moves[1, 0, 0] = torch.tensor(bad, dtype=torch.int32)
        counts = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
        pa.move_tokens(cache.k, cache.v, bt, lens, moves, counts, 40, cache.num_blocks)
        torch.cuda.synchronize()
        assert pa.device_error() == pa.DEVERR_BAD_SLOT
    bt[1, 2] = -1
    moves[1, 0, 0] = torch.tensor([35, 0], dtype=torch.int32)
    pa.move_tokens(cache.k, cache.v, bt, lens, moves, counts, 40, cache.num_blocks)
    torch.cuda.synchronize()
    assert pa.device_error() == pa.DEVERR_BAD_BLOCK
    for a, b in zip(cache.arrays(), before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------------------
# as they are used together
# ---------------------------------------------------------------------------

class Op:
    def __init__(self, **kw):
        self.__dict__.update(kw)


@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_a_run_with_forks_appends_attention_and_evictions(kv):
    """Two forks of one prompt and a third sequence decode for 40 steps under a
    budget: append, attend, accumulate, and evict whenever a sequence passes it.
    A host model keeps every sequence's tokens (their values as the cache holds
    them, weights and positions) and says what attention has to be."""
    H, Hkv, d, budget, sinks, recent = 8, 2, 64, 64, 4, 16
    gen = torch.Generator().manual_seed(3)

    def rows(n):
        return torch.randn((n, Hkv, d), generator=gen).to(torch.bfloat16)

    def held(x):
        if kv == "int4":
            return ref.values_int4(*ref.quantise_int4(x.float().numpy()))
        return x.double().numpy()

    cache = PagedKVCache(64, Hkv, d, kv)
    cache.pool.enable_prefix_cache(8)
    names, k0, v0 = {}, rows(83), rows(83)
    k1, v1 = rows(30), rows(30)
    cache.run_phase([Op(seq="a"), Op(seq="a", k=k0, v=v0), Op(seq="c"),
                     Op(seq="c", k=k1, v=v1)], names)
    cache.run_phase([Op(parent="a", child="b")], names)
    seqs = ["a", "b", "c"]
    # per sequence and KV head: K values, V values, weight, position of each slot
    def start(k, v):
        return [[held(k)[:, g], held(v)[:, g], np.zeros(len(k)), np.arange(len(k))]
                for g in range(Hkv)]
    model = {"a": start(k0, v0), "b": start(k0, v0), "c": start(k1, v1)}
    seen = {"a": 83, "b": 83, "c": 30}
    tw = cache.track_weights(seqs, 128)
    for step in range(40):
        news = {s: (rows(1), rows(1)) for s in seqs}
        q = torch.randn((3, H, d), generator=gen).to(torch.bfloat16)
        si = cache.prepare_step([Op(seq=s, k=news[s][0], v=news[s][1]) for s in seqs], names, q)
        out = cache.step(si, 0.125)
        cache.accumulate_step(si, tw, 0.125)
        got = out.double().cpu().numpy()
        for b, s in enumerate(seqs):
            seen[s] += 1
            for g, m in enumerate(model[s]):
                m[0] = np.vstack([m[0], held(news[s][0])[:, g]])
                m[1] = np.vstack([m[1], held(news[s][1])[:, g]])
                m[2], m[3] = np.append(m[2], 0), np.append(m[3], seen[s] - 1)
                p = ref.probabilities(q[b:b + 1, g * 4:g * 4 + 4].double().numpy(), m[0], 0.125)
                want = (p @ m[1])[0]
                assert np.abs(got[b, g * 4:g * 4 + 4] - want).max() <= 1.2e-3 * np.abs(m[1]).max()
                m[2] = m[2] + p.sum((0, 1))
                w = tw.scores[b, g, :len(m[2])].double().cpu().numpy()
                assert np.allclose(w, m[2], rtol=REL, atol=1e-7)
                m[2] = w                       # the device's own sums decide the order
        cache.evict(tw, names, budget, sinks, recent)
        for b, s in enumerate(seqs):
            n = min(budget, len(model[s][0][2]))
            assert cache.pool.seq_len(names[s]) == n
            for g, m in enumerate(model[s]):
                mv, _, _ = ref.select(m[2], m[3], len(m[2]), n, seen[s], sinks, recent)
                for x in m:
                    x[mv[:, 1]] = x[mv[:, 0]]
                model[s][g] = [x[:n] for x in m]
                pos = tw.positions[b, g, :n].cpu().numpy()
                real = np.where(pos < 0, seen[s] - n + np.arange(n), pos)
                assert np.array_equal(real, model[s][g][3])
                assert set(range(sinks)) <= set(real) and seen[s] - 1 in real
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    free, used, shared = cache.pool.stats()
    assert used == 12 and shared == 0      # three sequences of 64 tokens, no block shared
