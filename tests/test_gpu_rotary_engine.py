"""Rotary positions and prompt attention as the engine runs them: prompts enter a cache, are
attended from their rows, and decode steps follow, against plain 64-bit forms.

Tolerance, derived before the first run. The plain form takes what the library keeps exactly:
queries and keys as the 16-bit rows that rotation gives (tested bit for bit elsewhere) or as
the values that the cache holds. Prompts: as in the tests of prompt attention, (eps + 2.5e-4 +
2^-21) sum p |v| and half a step of the output. Decode steps over 16-bit caches compute in fp32
with weights split in two 16-bit parts: under 1e-4 max |v|, as the other tests hold them to; over
8- and 4-bit caches within 1e-2 (INT8) and (2^-11 + 6.2e-4) max |v| (INT4) of the values held."""
from types import SimpleNamespace as Op

import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import compressed, rotary as ref
from paged_kv_cache_154_gb300.engine import PagedKVCache, Rotary, rope_table

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def host(t):
    return t.float().cpu().numpy()


def attend(q, keys, values, scale):
    """float64 attention of one query [H, d] over keys [L, H_kv, d]."""
    out = np.zeros(q.shape)
    group = q.shape[0] // keys.shape[1]
    for h in range(q.shape[0]):
        s = keys[:, h // group] @ q[h] * scale
        w = np.exp(s - s.max())
        out[h] = (w / w.sum()) @ values[:, h // group]
    return out


def held(cache, seq):
    """K and V values [L, H_kv, d] that the cache holds of a sequence (an id of the pool)."""
    n = cache.pool.seq_len(seq)
    bt, _ = cache.pool.block_tables([seq], max(1, -(-n // 16)))
    kv = compressed.cache_values(cache)
    t = np.arange(n)
    return tuple(x[bt[0][t // 16], :, t % 16] for x in kv)


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("axes", [1, 3])
def test_prompts_then_steps(kv, axes):
    H, G, d, dtype = 8, 2, 128, torch.bfloat16
    rng = np.random.default_rng(len(kv) + axes)
    gen = torch.Generator().manual_seed(5)
    lens = {"a": 37, "b": 1, "c": 130}
    cache = PagedKVCache(64, G, d, kv, free_order=rng.permutation(64))
    axis = None if axes == 1 else torch.from_numpy((np.arange(d // 2) % 3).astype(np.uint8)).cuda()
    rotary = Rotary(rope_table(400, d), freq_axis=axis)
    tab = rotary.cos_sin.cpu().numpy()
    assert np.array_equal(tab, ref.table(400, d)) or np.abs(tab - ref.table(400, d)).max() < 2e-7
    names = {}
    cache.reserve([Op(seq=s) for s in lens], names)
    scale = d ** -0.5

    def rows(n, heads):
        return (torch.randn((n, heads, d), generator=gen) * 0.8).to(dtype)

    def step(runs, prompt, places):
        """One step of these runs: its output, and its rows' rotation in plain form."""
        ops = [Op(seq=s, k=rows(r, G), v=rows(r, G)) for s, r in runs.items()]
        q = rows(sum(runs.values()), H)
        pos = np.concatenate(places, -1).astype(np.int32)
        si = cache.prepare_step(ops, names, q.cuda(), rotary=rotary, prompt=prompt,
                                positions=None if axes == 1 else pos)
        out = cache.step(si, scale)
        assert pa.device_error() == 0
        if axes == 1:
            assert np.array_equal(si.positions.cpu().numpy().reshape(-1), pos.reshape(-1))
        c, s = ref.angles(tab, pos.reshape(axes, -1),
                          None if axis is None else axis.cpu().numpy())
        qr = torch.from_numpy(ref.rotate(host(q), c, s, False, np.float32)).to(dtype)
        key = torch.cat([op.k for op in ops])
        kr = torch.from_numpy(ref.rotate(host(key), c, s, False, np.float32)).to(dtype)
        assert torch.equal(si.q_rotated.cpu(), qr) and torch.equal(si.key_rotated.cpu(), kr)
        assert torch.equal(si.q.cpu(), q)
        return host(out), host(qr).astype(np.float64), host(kr), host(
            torch.cat([op.v for op in ops]))

    def places(run, first):
        t = first + np.arange(run)
        return np.stack([t // 12, t % 12 // 4, t % 4])[:axes] if axes > 1 else t[None]

    out, q, k, v = step(lens, True, [places(n, 0) for n in lens.values()])
    eps = torch.finfo(dtype).eps / 2
    want = ref.prompt_attention(q, k, v, list(lens.values()), scale)
    size = ref.prompt_attention(q, k, np.abs(v), list(lens.values()), scale)
    assert (np.abs(out - want) <= (eps + 2.6e-4) * size * (1 + eps) + eps * np.abs(want) + 1e-7).all()

    rel = {"bf16": 1e-4, "int8": 1e-2, "int4": 2.0 ** -11 + 6.2e-4}[kv]
    for i in range(3):
        runs = {"a": 1, "b": 1 + i, "c": 2}
        first = {s: cache.pool.seq_len(names[s]) for s in runs}
        out, q, _, _ = step(runs, False, [places(r, first[s]) for s, r in runs.items()])
        at = 0
        for s, r in runs.items():
            keys, values = held(cache, names[s])
            for j in range(r):
                n = first[s] + j + 1
                want = attend(q[at + j], keys[:n], values[:n], scale)
                assert np.abs(out[at + j] - want).max() <= rel * max(1.0, np.abs(values).max())
            at += r


def test_a_captured_step_runs_again():
    """A rotated step captured in a graph: replays do not rotate what is rotated already."""
    H, G, d = 4, 2, 64
    cache = PagedKVCache(16, G, d, "f16")
    names = {}
    cache.reserve([Op(seq=0), Op(seq=1)], names)
    gen = torch.Generator().manual_seed(9)

    def rows(n, heads):
        return torch.randn((n, heads, d), generator=gen).half()

    si = cache.prepare_step([Op(seq=0, k=rows(20, G), v=rows(20, G)),
                             Op(seq=1, k=rows(7, G), v=rows(7, G))], names, rows(27, H).cuda(),
                            rotary=Rotary(rope_table(64, 32), True), prompt=True)
    first = cache.step(si, 0.125).clone()
    kept = cache.k.clone()
    g = cache.capture(cache.step, si, 0.125)
    si.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(si.out, first) and torch.equal(cache.k, kept)


def test_positions_count_evicted_tokens():
    """After an eviction the next token's position is its place in the text."""
    H, G, d = 2, 1, 64
    cache = PagedKVCache(16, G, d, "bf16")
    names = {}
    cache.reserve([Op(seq=0)], names)
    gen = torch.Generator().manual_seed(3)

    def rows(n, heads):
        return torch.randn((n, heads, d), generator=gen).bfloat16()

    rotary = Rotary(rope_table(200, d))
    si = cache.prepare_step([Op(seq=0, k=rows(50, G), v=rows(50, G))], names, rows(50, H).cuda(),
                            rotary=rotary)
    cache.step(si, 0.125)
    tw = cache.track_weights([0], 64)
    cache.accumulate_step(si, tw, 0.125)
    cache.evict(tw, names, 20)
    si = cache.prepare_step([Op(seq=0, k=rows(2, G), v=rows(2, G))], names, rows(2, H).cuda(),
                            rotary=rotary)
    assert si.positions.tolist() == [50, 51]
    # the weights are those of the rotated queries
    cache.step(si, 0.125)
    before = tw.scores.clone()
    cache.accumulate_step(si, tw, 0.125)
    keys, _ = held(cache, names[0])
    want = np.zeros(22)
    for j in range(2):
        for h in range(H):
            s = keys[:21 + j, 0] @ host(si.q_rotated)[j, h].astype(np.float64) * 0.125
            w = np.exp(s - s.max())
            want[:21 + j] += w / w.sum()
    got = (tw.scores - before)[0, 0, :22].cpu().numpy()
    assert np.abs(got - want).max() < 1e-4


def test_long_prompts_take_a_workspace():
    """A prompt of more than 8192 tokens beside a short one, each the same as alone through the
    call itself; captured, it runs again on other rows."""
    H, G, d, lens = 2, 1, 64, [9000, 20]
    cache = PagedKVCache(600, G, d, "int8")
    names = {}
    cache.reserve([Op(seq=0), Op(seq=1)], names)
    gen = torch.Generator().manual_seed(10)

    def rows(n, heads):
        return torch.randn((n, heads, d), generator=gen).half()

    ops = [Op(seq=i, k=rows(n, G), v=rows(n, G)) for i, n in enumerate(lens)]
    si = cache.prepare_step(ops, names, rows(sum(lens), H).cuda(), prompt=True)
    assert si.workspace.nbytes == pa.prompt_attention_workspace_size(d, max(lens)) > 0
    si.workspace.fill_(255)

    def alone():
        parts = []
        for a, b in ((0, lens[0]), (lens[0], sum(lens))):
            out = torch.empty_like(si.q[a:b])
            start = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
            ws = torch.full_like(si.workspace, 255)
            pa.prompt_attention(out, si.q[a:b], si.key[a:b], si.value[a:b], start, b - a,
                                d ** -0.5, ws)
            parts.append(out)
        return torch.cat(parts)

    assert torch.equal(cache.step(si, d ** -0.5), alone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend_step(si, d ** -0.5)
    si.q.copy_(rows(sum(lens), H))
    si.out.fill_(float("nan"))
    graph.replay()
    assert torch.equal(si.out, alone())
    assert pa.device_error() == 0


def test_prompts_then_steps_fp8():
    """As above over an FP8 cache: codes of the rotated keys by per-head scales, and decode steps
    over them, whose products take bf16 queries and the codes exactly (as fp16) and weights
    rounded to fp16 once, by 2^-11 of themselves for the product and as much for their sum at
    most; scores as above, 2.6e-4 of a weight. Both act on at most max |v|."""
    H, G, d, dtype = 8, 2, 128, torch.bfloat16
    gen = torch.Generator().manual_seed(6)
    lens = {"a": 37, "b": 130}
    scales = np.array([0.011, 0.02], np.float32), np.array([0.013, 0.009], np.float32)
    cache = PagedKVCache(64, G, d, "fp8", head_scales=scales)
    rotary = Rotary(rope_table(400, d), interleaved=True)
    tab, names, scale = rotary.cos_sin.cpu().numpy(), {}, d ** -0.5
    cache.reserve([Op(seq=s) for s in lens], names)

    def rows(n, heads):
        return (torch.randn((n, heads, d), generator=gen) * 0.8).to(dtype)

    def step(runs, prompt):
        at = {s: cache.pool.seq_len(names[s]) for s in runs}
        ops = [Op(seq=s, k=rows(r, G), v=rows(r, G)) for s, r in runs.items()]
        si = cache.prepare_step(ops, names, rows(sum(runs.values()), H).cuda(), rotary=rotary,
                                prompt=prompt)
        out = host(cache.step(si, scale))
        assert pa.device_error() == 0
        pos = np.concatenate([at[s] + np.arange(r) for s, r in runs.items()])[None]
        c, s = ref.angles(tab, pos)
        q, k = (ref.rotate(host(x), c, s, True, np.float32) for x in (si.q, si.key))
        slots = si.slots.cpu().numpy()
        for got, x, z in ((cache.k, k, scales[0]), (cache.v, host(si.value), scales[1])):
            code = torch.from_numpy(x / z[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            got = got.view(torch.uint8).cpu().numpy()[slots // 16, :, slots % 16]
            assert np.array_equal(got, code.view(torch.uint8).numpy())
        q, k = (host(torch.from_numpy(x).to(dtype)) for x in (q, k))
        return out, q.astype(np.float64), k, host(si.value), at

    out, q, k, v, _ = step(lens, True)
    eps = torch.finfo(dtype).eps / 2
    want = ref.prompt_attention(q, k, v, list(lens.values()), scale)
    size = ref.prompt_attention(q, k, np.abs(v), list(lens.values()), scale)
    assert (np.abs(out - want) <= (eps + 2.6e-4) * size * (1 + eps) + eps * np.abs(want) + 1e-7).all()
    for i in range(2):
        runs = {"a": 1 + 2 * i, "b": 2}
        out, q, _, _, first = step(runs, False)
        at = 0
        for s, r in runs.items():
            n = cache.pool.seq_len(names[s])
            bt, _ = cache.pool.block_tables([names[s]], -(-n // 16))
            t = np.arange(n)
            keys, values = (x.float().cpu().numpy().astype(np.float64)[bt[0][t // 16], :, t % 16]
                            * z[:, None] for x, z in ((cache.k, scales[0]), (cache.v, scales[1])))
            for j in range(r):
                e = first[s] + j + 1
                want = attend(q[at + j], keys[:e], values[:e], scale)
                assert np.abs(out[at + j] - want).max() <= (2.0 ** -10 + 2.6e-4) * np.abs(values).max()
            at += r
