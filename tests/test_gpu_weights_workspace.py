"""Workspaces of the weight sums: one buffer, sized for a server's largest call, under
every smaller one, and the buffers of captured steps. Tolerances are those of
test_gpu_eviction."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import compressed as ref
from paged_kv_cache_154_gb300.engine import PagedKVCache
from test_gpu_eviction import REL, Op, check, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def size(S, H, Hkv, d, run, longest):
    return pa.accumulate_weights_workspace_size(S, S * run, H, Hkv, d, run, longest)


# the largest call: sequences, query heads, KV heads, head_dim, query run, tokens. In the
# first the stored logits of the largest call pass their limit by a token, in the second
# its query rows do, in the third they are stored.
LARGEST = [(64, 32, 8, 128, 1, 32769), (40, 64, 8, 64, 5, 8192), (9, 16, 2, 64, 2, 20000)]
SMALLER = [([1, 15, 16, 17, 100, 511, 512, 700], [1] * 8), ([4097], [1]), ([5000, 33], [1, 1]),
           ([900, 40], [2, 1]), ([6000, 5999, 6000, 6000, 5000], [1] * 5)]


@pytest.mark.parametrize("kv", ["bf16", "int4", "int8"])
@pytest.mark.parametrize("largest", LARGEST, ids=lambda x: f"{x[0]}x{x[5]}_run{x[4]}")
@pytest.mark.parametrize("case", SMALLER, ids=lambda c: f"{len(c[0])}x{max(c[0])}_run{max(c[1])}")
def test_a_buffer_for_the_largest_call_serves_the_smaller(largest, case, kv):
    lens, runs = case
    _, H, Hkv, d, run, _ = largest
    runs = [min(r, run) for r in runs]
    room = size(*largest)
    ws = torch.full((room + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    cache, tables, src = filled(5, kv, lens, Hkv, d)
    q = torch.randn((sum(runs), H, d), generator=torch.Generator().manual_seed(8)).to(src)
    qsl = np.concatenate([[0], np.cumsum(runs)]).astype(np.int32)
    out = torch.full((len(lens), Hkv, max(lens)), -7.0, device="cuda")
    pa.accumulate_weights(out, None, q.cuda(), cache.k, torch.from_numpy(tables).cuda(),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens),
                          d ** -0.5, None if max(runs) == 1 else torch.from_numpy(qsl).cuda(),
                          max(runs), cache.num_blocks, cache.k_scale, cache.k_zp, ws[:room])
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    assert (ws[room:] == 0xFF).all()
    check(out, cache, tables, lens, qsl, q, d ** -0.5, None, max(lens))


def test_a_buffer_too_small_for_the_call_is_refused():
    lens, H, Hkv, d = [700], 8, 2, 64
    cache, tables, src = filled(6, "bf16", lens, Hkv, d)
    q = torch.randn((1, H, d)).to(src).cuda()
    out = torch.zeros((1, Hkv, 700), device="cuda")
    least = 2 * 4 * 6 * 8 + 256 - 2 * 4 * 6 * 8 % 256    # sums of 6 tiles, to 256 bytes
    args = (cache.k, torch.from_numpy(tables).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), 700, 0.125, None, 1,
            cache.num_blocks, None, None)
    pa.accumulate_weights(out, None, q, *args, torch.empty(least, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pa.PAError, match="workspace"):
        pa.accumulate_weights(out, None, q, *args,
                              torch.empty(least - 1, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    check(out, cache, tables, lens, np.arange(2), q.cpu(), 0.125, None, 700)


def test_captured_steps_keep_their_workspaces():
    """Two captured steps of one batch's weights, the later and larger one in between: each
    replays into the buffer it was captured with, and the sums are those of eager steps."""
    H, Hkv, d = 8, 2, 64
    gen = torch.Generator().manual_seed(3)

    def rows(n):
        return torch.randn((n, Hkv, d), generator=gen).to(torch.bfloat16)

    cache, names = PagedKVCache(200, Hkv, d, "int4"), {}
    cache.run_phase([Op(seq="a"), Op(seq="a", k=rows(900), v=rows(900)), Op(seq="b"),
                     Op(seq="b", k=rows(33), v=rows(33))], names)
    tw = cache.track_weights(["a", "b"], 1000)
    steps, graphs, held = [], [], []
    for n in (1, 20):
        q = torch.randn((2 * n, H, d), generator=gen).to(torch.bfloat16)
        si = cache.prepare_step([Op(seq=s, k=rows(n), v=rows(n)) for s in ("a", "b")], names, q)
        cache.write_step(si)
        graphs.append(cache.capture(cache.accumulate_step, si, tw, 0.125))
        steps.append(si)
        held.append(si.weights_workspace.data_ptr())
    other = [torch.full((w.numel(),), 0x5A, dtype=torch.uint8, device="cuda")
             for w in (si.weights_workspace for si in steps) for _ in range(3)]
    tw.scores.zero_()
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    assert [si.weights_workspace.data_ptr() for si in steps] == held and held[0] != held[1]
    assert all((x == 0x5A).all() for x in other)
    k, _ = ref.cache_values(cache)
    want = 0
    for si, times in zip(steps, (2, 1)):
        lens, nq = si.context_lens.tolist(), si.q.shape[0]
        w = ref.weights(si.q.double().cpu().numpy(), k, si.block_tables.cpu().numpy(), lens,
                        np.arange(3) * (nq // 2), 0.125, 1000)
        want = want + times * w
    got = tw.scores.double().cpu().numpy()
    # three additions to a sum, each rounded by 2^-24
    assert (np.abs(got - want) <= (REL + 3 * 2.0 ** -24) * want + 1e-30).all()
