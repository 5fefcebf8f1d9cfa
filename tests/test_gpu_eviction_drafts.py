"""Weights and evictions of sequences whose draft tokens are partly taken back, against
a host model of every slot. Tolerances are those of test_gpu_eviction and
test_gpu_int4."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import compressed as ref
from paged_kv_cache_154_gb300.engine import PagedKVCache
from test_gpu_eviction import REL, Op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Model:
    """The slots of one sequence, per KV head [K values, V values, weights, positions]."""

    def __init__(self, kv, Hkv):
        self.kv, self.heads, self.seen = kv, [[None, None, np.zeros(0), np.zeros(0, int)]
                                              for _ in range(Hkv)], 0

    def held(self, x):
        if self.kv == "int4":
            return ref.values_int4(*ref.quantise_int4(x.float().numpy()))
        return x.double().numpy()

    def append(self, k, v):
        k, v = self.held(k), self.held(v)
        for g, m in enumerate(self.heads):
            for i, x in ((0, k), (1, v)):
                m[i] = x[:, g] if m[i] is None else np.vstack([m[i], x[:, g]])
            m[2] = np.append(m[2], np.zeros(len(k)))
            m[3] = np.append(m[3], self.seen + np.arange(len(k)))
        self.seen += len(k)

    def truncate(self, n):
        self.seen -= len(self) - n
        self.heads = [[x[:n] for x in m] for m in self.heads]

    def __len__(self):
        return len(self.heads[0][2])


@pytest.mark.parametrize("kv", ["bf16", "int4"])
@pytest.mark.parametrize("first", ["truncate", "accumulate"])
def test_rejected_drafts_leave_nothing_behind(kv, first):
    H, Hkv, d, budget, sinks, recent, scale = 8, 2, 64, 60, 4, 12, 0.125
    gen, rng = torch.Generator().manual_seed(5), np.random.default_rng(5)

    def rows(n, heads=Hkv):
        return torch.randn((n, heads, d), generator=gen).to(torch.bfloat16)

    cache, names, seqs = PagedKVCache(64, Hkv, d, kv), {}, ["a", "b", "c"]
    model = {s: Model(kv, Hkv) for s in seqs}
    for s, n in zip(seqs, (70, 15, 1)):
        k, v = rows(n), rows(n)
        cache.run_phase([Op(seq=s), Op(seq=s, k=k, v=v)], names)
        model[s].append(k, v)
    tw = cache.track_weights(seqs, 128)
    for step in range(30):
        runs = rng.integers(1, 6, 3)
        kept = np.array([rng.integers(0 if step % 3 else 1, r + 1) for r in runs])
        drafts = [(rows(r), rows(r)) for r in runs]
        q = rows(int(runs.sum()), H)
        si = cache.prepare_step([Op(seq=s, k=k, v=v) for s, (k, v) in zip(seqs, drafts)], names, q)
        got = cache.step(si, scale).double().cpu().numpy()
        for s, (k, v) in zip(seqs, drafts):
            model[s].append(k, v)
        lens = np.array([len(model[s]) for s in seqs])
        if first == "accumulate":
            cache.accumulate_step(si, tw, scale, kept)
        cache.truncate(tw, names, lens - (runs - kept))
        if first == "truncate":
            cache.accumulate_step(si, tw, scale, kept)
        at = 0
        for b, s in enumerate(seqs):
            r, n, a = runs[b], lens[b] - (runs[b] - kept[b]), kept[b]
            for g, m in enumerate(model[s].heads):
                queries = q[at:at + r, g * 4:g * 4 + 4].double().numpy()
                p = ref.probabilities(queries, m[0], scale)
                want = np.einsum("igt,td->igd", p, m[1])
                assert np.abs(got[at:at + r, g * 4:g * 4 + 4] - want).max() <= \
                    1.2e-3 * np.abs(m[1]).max()
                m[2] = m[2] + p[:a].sum((0, 1))
            at += r
            model[s].truncate(n)
            assert cache.pool.seq_len(names[s]) == n
            for g, m in enumerate(model[s].heads):
                w = tw.scores[b, g].double().cpu().numpy()
                assert np.allclose(w[:n], m[2], rtol=REL, atol=1e-7)
                assert not w[n:].any()
                m[2] = w[:n]               # the device's own sums decide the order
        if step % 4 == 3:
            over = np.array([len(model[s]) for s in seqs])
            cache.evict(tw, names, budget, sinks, recent)
            for b, s in enumerate(seqs):
                n = min(budget, over[b])
                for g, m in enumerate(model[s].heads):
                    mv, _, _ = ref.select(m[2], m[3], over[b], n, model[s].seen, sinks, recent)
                    for x in m:
                        x[mv[:, 1]] = x[mv[:, 0]]
                    model[s].heads[g] = [x[:n] for x in m]
                    pos = tw.positions[b, g, :n].cpu().numpy()
                    real = np.where(pos < 0, model[s].seen - n + np.arange(n), pos)
                    assert np.array_equal(real, model[s].heads[g][3])
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    assert (tw.evicted > 0).any()
    with pytest.raises(ValueError, match="eviction"):
        cache.truncate(tw, names, 1)


@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_a_batch_that_changes_keeps_its_weights(kv):
    """A sequence ends, another joins and one that was evicted from is forked; the rest
    come over into new weights. Sinks and recent tokens stay those of the text."""
    H, Hkv, d, budget, sinks, recent, scale = 8, 2, 64, 48, 4, 12, 0.125
    gen = torch.Generator().manual_seed(6)

    def rows(n, heads=Hkv):
        return torch.randn((n, heads, d), generator=gen).to(torch.bfloat16)

    cache, names, model = PagedKVCache(64, Hkv, d, kv), {}, {}

    def join(s, n):
        k, v = rows(n), rows(n)
        cache.run_phase([Op(seq=s), Op(seq=s, k=k, v=v)], names)
        model[s] = Model(kv, Hkv)
        model[s].append(k, v)

    def steps(seqs, tw, count):
        for _ in range(count):
            new = [(rows(1), rows(1)) for _ in seqs]
            q = rows(len(seqs), H)
            si = cache.prepare_step([Op(seq=s, k=k, v=v) for s, (k, v) in zip(seqs, new)], names,
                                    q)
            cache.write_step(si)
            cache.accumulate_step(si, tw, scale)
            for b, (s, (k, v)) in enumerate(zip(seqs, new)):
                model[s].append(k, v)
                for g, m in enumerate(model[s].heads):
                    p = ref.probabilities(q[b:b + 1, g * 4:g * 4 + 4].double().numpy(), m[0], scale)
                    m[2] = m[2] + p.sum((0, 1))
                    w = tw.scores[b, g].double().cpu().numpy()
                    assert np.allclose(w[:len(m[2])], m[2], rtol=REL, atol=1e-7)
                    m[2] = w[:len(m[2])]
            cache.evict(tw, names, budget, sinks, recent)
            for b, s in enumerate(seqs):
                L, n = len(model[s]), min(budget, len(model[s]))
                for g, m in enumerate(model[s].heads):
                    mv, _, _ = ref.select(m[2], m[3], L, n, model[s].seen, sinks, recent)
                    for x in m:
                        x[mv[:, 1]] = x[mv[:, 0]]
                    model[s].heads[g] = [x[:n] for x in m]
                    pos = tw.positions[b, g, :n].cpu().numpy()
                    real = np.where(pos < 0, model[s].seen - n + np.arange(n), pos)
                    assert np.array_equal(real, model[s].heads[g][3])
                    assert set(range(min(sinks, n))) <= set(real) and model[s].seen - 1 in real
        return tw

    for s, n in (("a", 70), ("b", 30), ("c", 45)):
        join(s, n)
    tw = steps(["a", "b", "c"], cache.track_weights(["a", "b", "c"], 96), 6)
    cache.pool.seq_free(names.pop("b"))
    join("d", 60)
    cache.run_phase([Op(parent="a", child="f")], names)
    twin = Model(kv, Hkv)
    twin.seen, twin.heads = model["a"].seen, [[x.copy() for x in m] for m in model["a"].heads]
    model["f"] = twin
    seqs = ["d", "c", "f", "a"]
    tw = cache.track_weights(seqs, 80, carry=[tw], parents={"f": "a"})
    steps(seqs, tw, 8)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
