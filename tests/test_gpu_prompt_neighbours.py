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


@pytest.mark.parametrize("group", [1, 3, 5, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_neighbours_with_other_scores(group, d, dt):
    """Rows of another prompt stand in the same tiles as a prompt's own (and are not written from
    there): their scores, small or large, do not decide how the prompt's are computed."""
    lens = [70, 40, 300, 9, 513, 150, 33, 77]
    at = np.concatenate([[0], np.cumsum(lens)])
    T = int(at[-1])
    q, k, v = rows(group + d, T, group, 1, d, DT[dt])
    q *= 3                                     # references move
    start = torch.from_numpy(at.astype(np.int32)).cuda()
    for bad in (1, 3, 5, 7):
        outs = []
        for factor in (1.0, 0.0, 8.0, -60.0):
            q2, k2, v2 = q.clone(), k.clone(), v.clone()
            part = slice(int(at[bad]), int(at[bad + 1]))
            q2[part] *= factor
            k2[part] *= factor
            v2[part] *= factor
            out = torch.zeros_like(q)
            pa.prompt_attention(out, q2, k2, v2, start, max(lens), d ** -0.5)
            outs.append(torch.cat((out[:part.start], out[part.stop:])))
        assert pa.device_error() == 0 and torch.isfinite(outs[0]).all()
        for o in outs[1:]:
            assert torch.equal(o, outs[0])
