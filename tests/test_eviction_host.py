"""The host side of eviction and of 4-bit caches, without a GPU: private copies
and truncation in the block pool, and the refusals of the device calls, which
are made before anything is launched."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_154_gb300 as pa
from oracle import compressed as ref


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()


def table(pool, seq):
    n = (pool.seq_len(seq) + 15) // 16
    return pool.block_tables([seq], max(1, n))[0][0, :n].tolist()


def test_private_copies_and_truncation():
    p = pa.Pool(20)
    a = p.seq_create()
    p.seq_append_slots(a, 70)                 # five blocks
    b = p.seq_fork(a)
    before = table(p, a)
    pairs = p.seq_make_private(b, 33)         # its first three
    assert pairs[:, 0].tolist() == before[:3]
    assert table(p, b) == pairs[:, 1].tolist() + before[3:]
    assert table(p, a) == before
    assert [p.refcount(x) for x in before] == [1, 1, 1, 2, 2]
    assert len(p.seq_make_private(b, 33)) == 0
    p.seq_truncate(b, 33)
    assert p.seq_len(b) == 33 and [p.refcount(x) for x in before] == [1] * 5
    p.seq_truncate(a, 16)
    assert p.stats() == (20 - 1 - 3, 4, 0)
    p.seq_truncate(a, 0)
    p.seq_free(a)
    p.seq_free(b)
    assert p.stats() == (20, 0, 0)


def test_truncation_takes_back_draft_tokens():
    p = pa.Pool(8)
    a = p.seq_create()
    s0, _ = p.seq_append_slots(a, 20)
    s1, _ = p.seq_append_slots(a, 14)
    p.seq_truncate(a, 23)
    s2, _ = p.seq_append_slots(a, 4)
    assert s2[:4].tolist() == s1[3:7].tolist()


def test_private_copies_are_all_or_nothing():
    p = pa.Pool(6)
    a = p.seq_create()
    p.seq_append_slots(a, 64)
    b = p.seq_fork(a)
    with pytest.raises(pa.PAError) as e:
        p.seq_make_private(b, 64)             # four copies, two blocks free
    assert e.value.status == 3
    assert p.stats() == (2, 4, 4) and table(p, b) == table(p, a)
    one, n = np.zeros((1, 2), np.int32), ctypes.c_int32()
    for out, room in ((one.ctypes.data, 1), (None, 9)):
        assert pa.lib().pa_seq_make_private(p._h, b, 32, out, room, ctypes.addressof(n)) == 1
        assert table(p, b) == table(p, a) and n.value == 0
    for bad in (-1, 65):
        with pytest.raises(pa.PAError):
            p.seq_make_private(b, bad)
        with pytest.raises(pa.PAError):
            p.seq_truncate(b, bad)
    for call in (p.seq_make_private, p.seq_truncate):
        with pytest.raises(pa.PAError):
            call(7, 0)
    assert pa.lib().pa_seq_truncate(None, 0, 0) == 1
    assert pa.lib().pa_seq_make_private(None, 0, 0, None, 0, ctypes.addressof(n)) == 1


def test_blocks_that_will_be_rewritten_leave_the_prefix_cache():
    p = pa.Pool(16)
    p.enable_prefix_cache(16)
    toks = list(range(100, 164))
    a, hit = p.create_with_prefix(toks)
    p.append_tokens(a, toks)                  # four registered blocks
    assert hit == 0 and p.prefix_stats()[1] == 4
    p.seq_make_private(a, 20)                 # two of them are about to be rewritten
    assert p.prefix_stats()[1] == 2
    b, hit = p.create_with_prefix(toks + [1])
    assert hit == 0                           # the chain starts with a rewritten block
    p.seq_truncate(a, 20)
    p.append_tokens(a, list(range(40)))       # no known prefix any more: nothing registered
    p.seq_free(a)
    c, hit = p.create_with_prefix(toks + [1])
    assert hit == 0


def test_a_shared_registered_block_keeps_serving_the_others():
    p = pa.Pool(16)
    p.enable_prefix_cache(16)
    toks = list(range(48))
    a, _ = p.create_with_prefix(toks)
    p.append_tokens(a, toks)
    b, hit = p.create_with_prefix(toks + [5])
    assert hit == 48
    pairs = p.seq_make_private(b, 48)
    assert len(pairs) == 3
    c, hit = p.create_with_prefix(toks + [5])
    assert hit == 48 and table(p, c) == table(p, a)


@pytest.mark.parametrize("cut", [5, 16, 23])
def test_a_truncated_block_is_not_handed_out_for_its_old_prefix(cut):
    p = pa.Pool(16)
    p.enable_prefix_cache(16)
    toks = list(range(32))
    a, _ = p.create_with_prefix(toks)
    p.append_tokens(a, toks)
    b = p.seq_fork(a)
    p.seq_truncate(a, cut)
    p.seq_free(b)
    p.seq_append_slots(a, 3)                  # overwrites slots of the cut block
    c, hit = p.create_with_prefix(toks + [9])
    # a whole block given up was not written again and still serves; a cut one does not
    assert hit == (32 if cut % 16 == 0 else cut // 16 * 16)
    assert not set(table(p, c)) & set(table(p, a)[cut // 16:])


@pytest.mark.parametrize("release", ["never", "before", "after"])
def test_a_cut_block_that_others_hold_keeps_serving(release):
    p = pa.Pool(16)
    p.enable_prefix_cache(16)
    toks = list(range(48))
    a, _ = p.create_with_prefix(toks)
    p.append_tokens(a, toks)
    b, hit = p.create_with_prefix(toks + [1])
    blocks = table(p, a)
    assert hit == 48 and table(p, b) == blocks
    p.seq_truncate(a, 23)                     # the second block is cut, but b has it whole
    c, hit = p.create_with_prefix(toks + [9])
    assert hit == 48 and table(p, c) == blocks
    p.seq_free(c)
    if release == "before":
        p.seq_free(b)                         # now a is its only holder
    _, pair = p.seq_append_slots(a, 3)        # into a copy while b has it, else in place
    assert (pair is None) == (release == "before")
    if release == "after":
        p.seq_free(b)
    d, hit = p.create_with_prefix(toks + [9])
    assert hit == (16 if release == "before" else 48)
    assert table(p, d)[1:] == ([] if release == "before" else blocks[1:])
    assert table(p, a)[0] == blocks[0] and (table(p, a)[1] == blocks[1]) == (release == "before")


def test_plain_selection_keeps_the_budget():
    """The plain form itself: the kept tokens by hand."""
    w = np.array([5, 1, 4, 4, 0, 9, 4], np.float32)
    none = np.full(7, -1)
    mv, s, pos = ref.select(w, none, 7, 3, 7, 0, 0)
    assert mv.tolist() == [[5, 1]] and s[:3].tolist() == [5, 9, 4] and pos[:3].tolist() == [0, 5, 2]
    mv, s, pos = ref.select(w, none, 7, 3, 7, 0, 1)      # slot 6 is recent
    assert mv.tolist() == [[5, 1], [6, 2]] and pos[:3].tolist() == [0, 5, 6]
    mv, s, pos = ref.select(w, none, 7, 2, 7, 1, 3)      # more protected than the budget
    assert mv.tolist() == [[4, 1]] and pos[:2].tolist() == [0, 4]


# ---------------------------------------------------------------------------
# refusals: fake, aligned addresses; the checks come before any launch
# ---------------------------------------------------------------------------

A, ODD = 0x10000, 0x10004


def refused(fn, args, **change):
    names = list(args)
    vals = [change.get(n, args[n]) for n in names]
    return getattr(pa.lib(), fn)(*vals)


WEIGHTS = dict(out=A, before=None, stride=64, q=A, qt=pa.PA_BF16, k=A, kt=pa.PA_INT4, ks=A, kz=A,
               bt=A, mb=4, cl=A, qsl=None, S=2, nq=2, mq=1, H=8, Hkv=2, d=64, bs=16, nb=9,
               scale=1.0, ml=64, ws=A, wb=1 << 30, st=None)


@pytest.mark.parametrize("change,status", [
    (dict(out=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(bt=None), 1),
    (dict(cl=None), 1), (dict(ks=None), 1), (dict(kz=None), 1), (dict(stride=63), 1),
    (dict(d=96), 2), (dict(bs=32), 2), (dict(H=7), 1), (dict(qt=pa.PA_F32), 2),
    (dict(kt=pa.PA_F16), 2), (dict(kt=9), 1), (dict(mb=3), 1), (dict(ml=0), 1), (dict(nq=3), 1),
    (dict(ws=None), 1), (dict(wb=64), 1), (dict(ws=A + 16), 1), (dict(out=ODD), 1),
    (dict(q=ODD), 1), (dict(k=ODD), 1), (dict(before=A + 2), 1), (dict(S=-1), 1),
    (dict(qsl=A, mq=1025, nq=2000, ml=2000, mb=125, stride=2000), 2), (dict(kz=A + 4), 1),
    (dict(S=65536, nq=65536), 2), (dict(nb=0), 1),
    (dict(ml=(1 << 30) + 1, mb=1 << 27, stride=1 << 31), 2),
    (dict(qsl=A, S=65535, nq=65535, H=32768, Hkv=32768, mq=64, ml=1 << 30, mb=1 << 27,
          stride=1 << 31), 2),
])
def test_weights_refusals(change, status):
    assert refused("pa_accumulate_weights", WEIGHTS, **change) == status
    assert pa.lib().pa_last_error()


SELECT = dict(moves=A, mm=32, counts=A, wo=A, po=A, w=A, pos=A, stride=64, cl=A, nl=A, tl=A, S=2,
              Hkv=2, ml=64, sinks=0, recent=0, st=None)


@pytest.mark.parametrize("change,status", [
    (dict(moves=None), 1), (dict(counts=None), 1), (dict(wo=None), 1), (dict(po=None), 1),
    (dict(w=None), 1), (dict(cl=None), 1), (dict(nl=None), 1), (dict(mm=31), 1),
    (dict(mm=0, ml=1), 1), (dict(stride=63), 1), (dict(ml=0), 1), (dict(sinks=-1), 1),
    (dict(recent=-1), 1), (dict(Hkv=0), 1), (dict(moves=A + 4), 1), (dict(S=65536), 2),
    (dict(S=-1), 1), (dict(ml=(1 << 30) + 1, mm=1 << 30, stride=1 << 31), 2),
])
def test_select_refusals(change, status):
    assert refused("pa_evict_select", SELECT, **change) == status


MOVE = dict(k=A, v=A, kt=pa.PA_INT4, ks=A, vs=A, kz=A, vz=A, bt=A, mb=4, cl=A, moves=A, mm=32,
            counts=A, S=2, Hkv=2, d=64, bs=16, nb=9, ml=64, st=None)


@pytest.mark.parametrize("change,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1), (dict(moves=None), 1),
    (dict(counts=None), 1), (dict(cl=None), 1), (dict(vz=None), 1), (dict(ks=None), 1),
    (dict(kt=pa.PA_FP8_E4M3, ks=None), 1), (dict(kt=pa.PA_F32), 1), (dict(d=32), 2),
    (dict(bs=8), 2), (dict(nb=0), 1), (dict(mb=3), 1), (dict(ml=0), 1), (dict(mm=0), 1),
    (dict(k=ODD), 1), (dict(v=ODD), 1), (dict(ks=A + 2), 1), (dict(moves=A + 4), 1),
    (dict(S=65536), 2), (dict(S=-1), 1), (dict(ml=(1 << 30) + 1, mb=1 << 27), 2),
])
def test_move_refusals(change, status):
    assert refused("pa_move_tokens", MOVE, **change) == status


GATHER = dict(key=A, value=A, ot=pa.PA_F32, k=A, v=A, kt=pa.PA_INT4, ks=A, vs=A, kz=A, vz=A,
              slots=A, T=4, nb=9, Hkv=2, d=64, bs=16, st=None)


@pytest.mark.parametrize("change,status", [
    (dict(key=None), 1), (dict(value=None), 1), (dict(slots=None), 1), (dict(ot=pa.PA_INT8), 2),
    (dict(kz=None), 1), (dict(T=-1), 1), (dict(key=ODD), 1), (dict(v=ODD), 1), (dict(d=256), 2),
    (dict(nb=0), 1),
])
def test_gather_refusals(change, status):
    assert refused("pa_gather_kv", GATHER, **change) == status


def test_int4_refusals_of_the_calls_that_were_there():
    L = pa.lib()
    append = dict(key=A, value=A, st=pa.PA_BF16, k=A, v=A, kt=pa.PA_INT4, ks=A, vs=A, kz=A, vz=A,
                  slots=A, T=4, nb=9, Hkv=2, d=64, bs=16, stream=None)
    for change in (dict(ks=None), dict(vz=None), dict(ks=A + 2)):
        assert refused("pa_append_kv", append, **change) == 1
    copy = dict(k=A, v=A, ks=A, vs=A, kz=A, vz=A, pairs=A, n=1, nb=9, Hkv=2, d=64, bs=16,
                kt=pa.PA_INT4, stream=None)
    for change in (dict(ks=None), dict(kz=A + 8)):
        assert refused("pa_copy_blocks", copy, **change) == 1
    ws = pa.decode_workspace_size(2, 2, 8, 2, 64, 1, 64)
    dec = dict(out=A, ot=pa.PA_F32, q=A, qt=pa.PA_BF16, k=A, v=A, kt=pa.PA_INT4, ks=A, vs=A, kz=A,
               vz=A, bt=A, mb=4, cl=A, qsl=None, S=2, nq=2, mq=1, H=8, Hkv=2, d=64, bs=16, nb=9,
               scale=1.0, ml=64, P=0, ws=A, wb=ws, stream=None)
    assert refused("pa_decode", dec, kz=None) == 1
    assert refused("pa_decode", dec, vs=A + 4) == 1
    assert refused("pa_decode", dec, P=32, wb=1 << 30) == 2
    assert refused("pa_decode", dec, nb=1 << 30) == 2            # 2^31 tiles
    assert refused("pa_decode", dec, qsl=A, H=4096, Hkv=4096, S=8192, nq=1 << 20, mq=64,
                   ml=64, wb=1 << 40) == 2                       # 2^31 rows of queries


def test_empty_calls_are_accepted():
    for fn, args, zero in (("pa_accumulate_weights", WEIGHTS, dict(S=0)),
                           ("pa_evict_select", SELECT, dict(S=0)),
                           ("pa_move_tokens", MOVE, dict(S=0)),
                           ("pa_gather_kv", GATHER, dict(T=0))):
        assert refused(fn, args, **zero) == 0


def test_workspace_sizes():
    f = pa.accumulate_weights_workspace_size
    assert f(0, 1, 8, 2, 64, 1, 64) == 0 and f(2, 2, 7, 2, 64, 1, 64) == 0
    # larger than a call may be, whatever the products of the sizes come to
    assert f(1, 1, 1 << 20, 1, 64, 1 << 20, 16) == 0 and f(1, 1, 8, 8, 64, 4097, 4097) == 0
    assert f(65535, 65535, 65535, 65535, 64, 16, 1 << 30) == 0
    assert f(1 << 30, 1 << 30, 8, 8, 64, 1, 64) == 0
    # 4 rows a KV head: the tiles' sums, and 16 bytes a token of logits
    logits = 2 * 2 * 608 * 16
    assert logits < f(2, 2, 8, 2, 64, 1, 600) < 1.1 * logits
    # more rows than are stored: sums of the rows' tiles alone, not 8 bytes a row and token
    assert 0 < f(2, 64, 8, 2, 64, 32, 600) < 2 * 2 * 128 * 600


def test_engine_refuses_evictions_before_anything_moves():
    from paged_kv_cache_154_gb300.engine import PagedKVCache
    cache = PagedKVCache(8, 2, 64, "bf16", device="cpu")     # nothing below reaches a GPU
    names = {}
    for name, n in (("a", 40), ("b", 20)):
        names[name] = cache.pool.seq_create()
        cache.pool.seq_append_slots(names[name], n)
    before = cache.pool.stats()
    tw = cache.track_weights(["a", "b"], 40)
    with pytest.raises(ValueError, match="negative"):
        cache.evict(tw, names, [10, -1])
    with pytest.raises(ValueError, match="twice"):
        cache.evict(cache.track_weights(["a", "a"], 40), names, 10)
    with pytest.raises(ValueError, match="holds 40 tokens"):
        cache.evict(cache.track_weights(["a", "b"], 39), names, 10)
    with pytest.raises(KeyError):
        cache.evict(cache.track_weights(["c"], 40), names, 10)
    cache.evict(tw, names, 40)                               # nothing is over its budget
    assert [cache.pool.seq_len(i) for i in names.values()] == [40, 20]
    assert cache.pool.stats() == before and not tw.evicted.any()


def cpu_engine(**lens):
    """An engine whose tensors are the host's (nothing reaches a GPU) with sequences of these
    lengths, and weights of 128 tokens each in which slot t has t + 1."""
    import torch
    from paged_kv_cache_154_gb300.engine import PagedKVCache
    cache, names = PagedKVCache(40, 2, 64, "bf16", device="cpu"), {}
    for name, n in lens.items():
        names[name] = cache.pool.seq_create()
        cache.pool.seq_append_slots(names[name], n)
    tw = cache.track_weights(list(lens), 128)
    for row, n in enumerate(lens.values()):
        tw.scores[row, :, :n] = torch.arange(1.0, n + 1)
    return cache, names, tw


def test_truncated_tokens_leave_no_weight():
    import torch
    cache, names, tw = cpu_engine(a=60, b=40, c=33)
    tw.positions[2, :, :33] = torch.arange(33)
    cache.truncate(tw, names, [57, 40, 20])
    assert [cache.pool.seq_len(i) for i in names.values()] == [57, 40, 20]
    for row, n in enumerate((57, 40, 20)):
        assert torch.equal(tw.scores[row, :, :n], torch.arange(1.0, n + 1).expand(2, n))
        assert not tw.scores[row, :, n:].any()
    assert torch.equal(tw.positions[2, :, :20], torch.arange(20).int().expand(2, 20))
    assert (tw.positions[2, :, 20:] == -1).all() and (tw.positions[:2] == -1).all()
    cache.truncate(tw, names, 50)
    assert [cache.pool.seq_len(i) for i in names.values()] == [50, 40, 20]
    assert not tw.scores[0, :, 50:].any() and tw.scores[0, 0, 49] == 50


def test_truncation_refusals():
    cache, names, tw = cpu_engine(a=60, b=40)
    tw.settled[:] = 32, 0                # as after an eviction that left 32 of a's tokens
    for lens, text in (([31, 40], "cut"), ([60, -1], "negative"), (0, "cut")):
        with pytest.raises(ValueError, match=text):
            cache.truncate(tw, names, lens)
        assert [cache.pool.seq_len(i) for i in names.values()] == [60, 40]
        assert tw.scores[0, 0, 59] == 60
    cache.truncate(tw, names, [32, 0])
    assert [cache.pool.seq_len(i) for i in names.values()] == [32, 0]


def test_accepted_queries_are_within_their_runs():
    from types import SimpleNamespace
    cache, names, tw = cpu_engine(a=60, b=40)
    si = SimpleNamespace(q=None, context_lens=None, query_start_loc=None, q_lens=[3, 1], seqs=None)
    for bad in ([4, 0], [3], [-1, 1], [2, 2]):
        with pytest.raises(ValueError, match="accepted"):
            cache.accumulate_step(si, tw, 0.125, bad)


def test_weights_come_over_when_the_batch_changes():
    import torch
    cache, names, tw = cpu_engine(a=60, b=40)
    tw.positions[0, :, :32] = torch.randperm(32).int()
    tw.evicted[0] = cache.pool.evicted[names["a"]] = 28     # as after an eviction of a
    tw.settled[0] = 32
    names["f"] = cache.pool.seq_fork(names["a"])
    names["n"] = cache.pool.seq_create()
    for seqs in (["a"], ["f"], ["n", "a"]):     # a fork has its parent's tokens
        for call in (lambda t: cache.evict(t, names, 8), lambda t: cache.truncate(t, names, 50)):
            with pytest.raises(ValueError, match="lost 28 tokens to evictions, 0 in these"):
                call(cache.track_weights(seqs, 128))
    assert cache.pool.seq_len(names["a"]) == 60
    new = cache.track_weights(["n", "f", "b", "a"], 100, carry=[tw], parents={"f": "a"})
    assert new.evicted.tolist() == [0, 28, 0, 28] and new.settled.tolist() == [0, 32, 0, 32]
    for i, j in ((1, 0), (2, 1), (3, 0)):
        assert torch.equal(new.scores[i], tw.scores[j, :, :100])
        assert torch.equal(new.positions[i], tw.positions[j, :, :100])
    assert not new.scores[0].any() and (new.positions[0] == -1).all()
    cache.truncate(new, names, 50)              # known to all of them
    new.scores[3] = 9
    assert tw.scores[0, 0, 5] == 6              # rows of its own
    cache.pool.seq_free(names["f"])
    assert names["f"] not in cache.pool.evicted and names["a"] in cache.pool.evicted


def test_a_step_of_other_sequences_is_refused():
    from types import SimpleNamespace
    cache, names, tw = cpu_engine(a=60, b=40)
    si = SimpleNamespace(q=None, context_lens=None, query_start_loc=None, q_lens=[1, 1],
                         seqs=["b", "a"])
    with pytest.raises(ValueError, match="weights of"):
        cache.accumulate_step(si, tw, 0.125)


def test_validation_without_host_memory_is_an_error():
    """PA_VALIDATE copies a call's slots to the host: where they do not fit, the call
    returns. In a process of its own that sees no GPU."""
    import os
    import subprocess
    import sys
    code = ("import resource, paged_kv_cache_154_gb300 as pa\n"
            "lib = pa.lib()\n"
            "now = int(open('/proc/self/statm').read().split()[0]) * resource.getpagesize()\n"
            "resource.setrlimit(resource.RLIMIT_AS, (now + (1 << 30),) * 2)\n"
            f"s = lib.pa_gather_kv(*{list(dict(GATHER, T=(1 << 31) - 1).values())!r})\n"
            "print(s, lib.pa_last_error().decode())\n")
    env = dict(os.environ, PA_VALIDATE="1", CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("1 ") and "host memory" in r.stdout, r.stdout
