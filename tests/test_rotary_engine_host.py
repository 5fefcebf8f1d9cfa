"""Rotary steps of the engine without a GPU: positions that the table of angles does not have are
refused, and the pool is as it was."""
from types import SimpleNamespace as Op

import numpy as np
import pytest
import torch

from paged_kv_cache_154_gb300.engine import PagedKVCache, Rotary, rope_table


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()


def rows(n, heads):
    return torch.zeros((n, heads, 64), dtype=torch.float16)


def op(seq, n):
    return Op(seq=seq, k=rows(n, 1), v=rows(n, 1))


@pytest.fixture
def cache():
    c = PagedKVCache(16, 1, 64, "f16", device="cpu")
    c.names = {}
    c.reserve([Op(seq="a"), Op(seq="b")], c.names)
    return c


ROTARY = Rotary(rope_table(40, 64, device="cpu"))


def test_positions_past_the_table(cache):
    cache.pool.seq_append_slots(cache.names["b"], 39)
    stats = cache.pool.stats()
    for runs in ({"a": 41}, {"a": 1, "b": 2}, {"b": 2, "a": 5}):
        with pytest.raises(ValueError, match="table of angles has 40"):
            cache.prepare_step([op(s, n) for s, n in runs.items()], cache.names,
                               rows(sum(runs.values()), 2), rotary=ROTARY)
    with pytest.raises(ValueError, match="position 40"):      # the same sequence twice
        cache.prepare_step([op("b", 1), op("b", 1)], cache.names, rows(2, 2), rotary=ROTARY)
    assert cache.pool.stats() == stats and cache.pool.seq_len(cache.names["a"]) == 0
    si = cache.prepare_step([op("a", 40), op("b", 1)], cache.names, rows(41, 2), rotary=ROTARY)
    assert si.positions.tolist() == [*range(40), 39]


def test_a_sequence_without_new_tokens_may_be_longer(cache):
    cache.pool.seq_append_slots(cache.names["b"], 50)
    si = cache.prepare_step([op("a", 2), op("b", 0)], cache.names, rows(2, 2), rotary=ROTARY)
    assert si.positions.tolist() == [0, 1]


def test_evicted_tokens_count(cache):
    cache.pool.seq_append_slots(cache.names["a"], 10)
    cache.pool.evicted[cache.names["a"]] = 30
    with pytest.raises(ValueError, match="'a' reaches position 40"):
        cache.prepare_step([op("a", 1)], cache.names, rows(1, 2), rotary=ROTARY)


@pytest.mark.parametrize("bad", [
    [0, 1], [0, 1, 2, 3], [[0, 1, 2], [0, 1, 40]], [0, -1, 2], [0, 1, (1 << 32) + 2],
    np.array([[0, 1, 40]]), torch.tensor([0, 1, 40]), torch.tensor(5), np.zeros((1, 1, 3), int)],
    ids=str)
def test_positions_given(cache, bad):
    with pytest.raises(ValueError, match="positions"):
        cache.prepare_step([op("a", 3)], cache.names, rows(3, 2), rotary=ROTARY, positions=bad)
    assert cache.pool.seq_len(cache.names["a"]) == 0


def test_positions_within(cache):
    for good in ([39, 0, 5], np.array([[39, 0, 5], [1, 2, 3]]), torch.tensor([39, 0, 5])):
        si = cache.prepare_step([op("a", 3)], cache.names, rows(3, 2), rotary=ROTARY,
                                positions=good)
        assert si.positions.dtype is torch.int32
        assert np.array_equal(si.positions.numpy(), np.asarray(good))
