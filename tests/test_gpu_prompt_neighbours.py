"""Nothing of one prompt reaches another's rows, with as many query heads per KV head as a call
takes: with more than 16 a chunk of a prompt is fewer tokens than the 16 keys that a product
takes at a time, so that products of several of a prompt's chunks pass its end. Equal bit for
bit, so there is no tolerance."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def rows(seed, T, H, G, d, dtype):
    gen = torch.Generator().manual_seed(seed)
    return tuple(torch.randn((T, n, d), generator=gen).to(dtype).cuda() for n in (H, G, G))


@pytest.mark.parametrize("group", [1, 16, 17, 43, 71, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_neighbours_that_are_not_finite(group, d, dt):
    """Prompts of 1 to 35 tokens (their chunks end at every residue of 16) and some that end
    about the edges of key tiles, between prompts of NaN and infinities, and such rows behind
    the last one: as beside finite ones."""
    G = 2 if group < 128 else 1
    good = list(range(1, 36)) + [111, 113, 127, 129, 143, 257]
    lens = [n for i, g in enumerate(good) for n in (g, 1 + i % 19)]
    lens[-1] = 0                                # the last good one ends at the rows behind
    at = np.concatenate([[0], np.cumsum(lens)])
    T = int(at[-1]) + 18
    q, k, v = rows(group + d, T, G * group, G, d, DT[dt])
    start = torch.from_numpy(at.astype(np.int32)).cuda()
    bad = torch.ones(T, dtype=torch.bool)
    for i in range(0, len(lens), 2):
        bad[at[i]:at[i + 1]] = False
    bad = bad.cuda()
    outs = []
    for fill in (None, (float("nan"), float("inf")), (float("-inf"), float("nan"))):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        if fill:
            q2[bad], k2[bad], v2[bad] = fill[0], fill[1], fill[0]
        out = torch.zeros_like(q)
        pa.prompt_attention(out, q2, k2, v2, start, max(lens), d ** -0.5)
        assert pa.device_error() == 0
        outs.append(out[~bad])
        assert (out[int(at[-1]):] == 0).all()
    assert torch.isfinite(outs[0]).all()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
