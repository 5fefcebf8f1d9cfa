"""Attention over prompts without a GPU: refusals of pa_prompt_attention and of its binding,
and the plain form against torch's."""
import struct

import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import rotary as ref


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()


A, ODD = 0x10000, 0x10004
CALL = dict(out=A, os=1024, q=A, qs=1024, k=A, ks=256, v=A, vs=256, dt=pa.PA_BF16, start=A, S=2,
            T=9, ml=8, H=8, G=2, d=128, scale=0.1, ws=None, wb=0, st=None)


def status(**change):
    """The call's status, which the packed form of it shares."""
    values = [change.get(n, CALL[n]) for n in CALL]
    got = pa.lib().pa_prompt_attention(*values)
    words = struct.pack("16qd3q", *[v or 0 for v in values])
    assert pa.lib().pa_prompt_attention_packed(words) == got
    return got


@pytest.mark.parametrize("change,want", [
    (dict(S=-1), 1), (dict(T=-1), 1), (dict(out=None), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(start=None), 1), (dict(dt=pa.PA_F32), 2), (dict(d=96), 2),
    (dict(H=7), 1), (dict(G=0), 1), (dict(H=0), 1), (dict(H=129, G=1, qs=1 << 20, os=1 << 20), 2),
    (dict(ml=0), 1), (dict(ml=(1 << 22) + 1), 2), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=3e38), 1),
    (dict(H=65536, G=65536, qs=1 << 30, os=1 << 30, ks=1 << 30, vs=1 << 30), 2),
    (dict(scale=float("inf")), 1), (dict(out=ODD), 1), (dict(q=ODD), 1), (dict(k=ODD), 1), (dict(v=ODD), 1), (dict(qs=1016), 1), (dict(os=1028), 1),
    (dict(ks=248), 1), (dict(vs=-256), 1), (dict(ks=1 << 38), 2), (dict(ws=ODD, wb=1 << 30), 1),
    (dict(ws=A, wb=1024, ml=8193), 1), (dict(ml=(1 << 19) + 1), 1),
    (dict(dt=pa.PA_F16, ml=(1 << 16) + 1), 1)])
def test_refusals(change, want):
    assert status(**change) == want
    assert pa.lib().pa_last_error()


def test_empty_calls_are_accepted():
    assert status(S=0, q=None) == 0
    assert status(T=0, q=None) == 0


def test_workspace_size():
    assert pa.prompt_attention_workspace_size(128, 8192) == 0
    assert pa.prompt_attention_workspace_size(96, 9000) == 0
    assert pa.prompt_attention_workspace_size(64, (1 << 22) + 1) == 0
    for d in (64, 128):
        assert pa.prompt_attention_workspace_size(d, 8193) == 152 * 2 * 128 * (d + 1) * 4


def test_binding():
    T, H, G, D = 6, 4, 2, 64
    b = torch.bfloat16

    def args(**change):
        return {**dict(out=torch.zeros((T, H, D), dtype=b), q=torch.zeros((T, H, D), dtype=b),
                       key=torch.zeros((T, G, D), dtype=b), value=torch.zeros((T, G, D), dtype=b),
                       seq_start=torch.zeros(3, dtype=torch.int32), max_seq_len=4, scale=0.1),
                **change}

    for name, wrong in (("out", torch.zeros((T, H, D))), ("key", torch.zeros((T + 1, G, D), dtype=b)),
                        ("value", torch.zeros((T, G, 2 * D), dtype=b)),
                        ("heads", None), ("seq_start", torch.zeros(3, dtype=torch.int64)),
                        ("seq_start", torch.zeros((1, 3), dtype=torch.int32))):
        change = {"value": torch.zeros((T, G + 1, D), dtype=b)} if wrong is None else {name: wrong}
        with pytest.raises(ValueError, match=name):
            pa.prompt_attention(**args(**change))
    with pytest.raises(ValueError, match="current device"):
        pa.prompt_attention(**args())


def test_plain_form_is_torchs():
    rng = np.random.default_rng(0)
    lens, H, G, d = [5, 0, 1, 33], 6, 3, 16
    T = sum(lens) + 2
    q, k, v = (rng.standard_normal((T, n, d)) for n in (H, G, G))
    got = ref.prompt_attention(q, k, v, lens, 0.3)
    at = 0
    for n in lens:
        x = [torch.from_numpy(a[at:at + n]).transpose(0, 1) for a in (q, k, v)]
        x[1:] = [t.repeat_interleave(H // G, 0) for t in x[1:]]
        if n:
            want = torch.nn.functional.scaled_dot_product_attention(*x, is_causal=True, scale=0.3)
            assert np.abs(got[at:at + n] - want.transpose(0, 1).numpy()).max() < 1e-12
        at += n
    assert (got[at:] == 0).all()
