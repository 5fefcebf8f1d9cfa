"""Rotary positions without a GPU: the refusals of pa_rope and pa_rope_append_kv, made
before anything is launched, the binding's own, and the plain forms against closed ones."""
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


# fake, aligned addresses: the checks come before any launch
A, ODD = 0x10000, 0x10004
ROPE = dict(qo=A, qos=1024, q=A, qs=1024, H=8, ko=A, kos=256, k=A, ks=256, G=2, dt=pa.PA_BF16,
            tab=A, most=64, rd=128, il=0, pos=A, axes=1, axis=None, inv=0, T=4, d=128, st=None)
APPEND = dict(qo=A, qos=1024, q=A, qs=1024, H=8, ko=None, kos=0, k=A, ks=256, v=A, vs=256,
              dt=pa.PA_BF16, kc=A, vc=A, kt=pa.PA_BF16, kscale=A, vscale=A, kzp=A, vzp=A, slots=A,
              tab=A, most=64, rd=128, il=0, pos=A, axes=1, axis=None, T=4, nb=9, G=2, d=128, bs=16,
              st=None)
BOTH = [
    (dict(T=-1), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(tab=None), 1),
    (dict(pos=None), 1), (dict(q=ODD), 1), (dict(qo=ODD), 1), (dict(k=ODD), 1), (dict(tab=ODD), 1),
    (dict(qs=1023), 1), (dict(qs=1016), 1), (dict(qos=1016), 1), (dict(ks=248), 1),
    (dict(ks=260), 1), (dict(qs=-1024), 1), (dict(d=96), 2), (dict(d=256), 2), (dict(rd=0), 2),
    (dict(rd=24), 2), (dict(rd=144), 2), (dict(d=64, rd=80), 2), (dict(most=0), 1),
    (dict(axes=0), 2), (dict(axes=5), 2), (dict(axes=2), 1), (dict(axes=2, axis=ODD), 1), (dict(dt=pa.PA_F32), 2),
    (dict(H=-1), 1), (dict(qos=2048), 1),
]


def status(fn, args, change):
    """The call's status, which the packed form of it shares."""
    values = [change.get(n, args[n]) for n in args]
    got = getattr(pa.lib(), fn)(*values)
    message = pa.lib().pa_last_error()
    words = struct.pack(f"{len(values)}q", *[v or 0 for v in values])
    assert getattr(pa.lib(), fn + "_packed")(words) == got
    assert pa.lib().pa_last_error() == message
    return got


@pytest.mark.parametrize("change,want", BOTH + [
    (dict(ko=None), 1), (dict(ko=ODD), 1), (dict(kos=248), 1), (dict(kos=512), 1), (dict(G=-1), 1)])
def test_rope_refusals(change, want):
    assert status("pa_rope", ROPE, change) == want
    assert pa.lib().pa_last_error()


@pytest.mark.parametrize("change,want", BOTH + [
    (dict(v=None), 1), (dict(kc=None), 1), (dict(slots=None), 1), (dict(kt=pa.PA_F16), 2),
    (dict(kt=pa.PA_INT8, kzp=None), 1), (dict(kt=pa.PA_INT4, vscale=None), 1),
    (dict(kt=pa.PA_FP8_E4M3, kscale=None), 1), (dict(kt=9), 1), (dict(nb=0), 1), (dict(bs=8), 2),
    (dict(G=0), 1), (dict(v=ODD), 1), (dict(vs=128), 1), (dict(vc=ODD), 1), (dict(ko=ODD), 1),
    (dict(ko=A, kos=512), 1), (dict(ko=A + 4096, kos=128), 1)])
def test_rope_append_refusals(change, want):
    assert status("pa_rope_append_kv", APPEND, change) == want


def test_packed_calls_need_their_array():
    for fn in ("pa_rope", "pa_rope_append_kv", "pa_prompt_attention"):
        assert getattr(pa.lib(), fn + "_packed")(None) == 1


def test_empty_calls_are_accepted():
    assert status("pa_rope", ROPE, dict(T=0, q=None)) == 0
    assert status("pa_rope", ROPE, dict(H=0, G=0, q=None, k=None)) == 0
    assert status("pa_rope_append_kv", APPEND, dict(T=0, k=None)) == 0


T, H, G, D, NB = 4, 6, 3, 64, 5


def rope_args():
    return dict(q_out=torch.zeros((T, H, D), dtype=torch.bfloat16),
                q=torch.zeros((T, H, D), dtype=torch.bfloat16),
                k_out=torch.zeros((T, G, D), dtype=torch.bfloat16),
                k=torch.zeros((T, G, D), dtype=torch.bfloat16), cos_sin=torch.zeros((9, D)),
                positions=torch.zeros(T, dtype=torch.int32))


def append_args():
    a = rope_args()
    return dict(q_out=a["q_out"], q=a["q"], key=a["k"], value=a["k_out"],
                k_cache=torch.zeros((NB, G, 16, D), dtype=torch.bfloat16),
                v_cache=torch.zeros((NB, G, 16, D), dtype=torch.bfloat16),
                slot_mapping=torch.zeros(T, dtype=torch.int64), cos_sin=a["cos_sin"],
                positions=a["positions"])


def refuses(match, fn, args, **change):
    with pytest.raises(ValueError, match=match):
        fn(**{**args, **change})


def test_binding_of_rope():
    b = torch.bfloat16
    for name in ("q_out", "k_out", "k"):
        refuses(name, pa.rope, rope_args(), **{name: torch.zeros((T + 1, H, D), dtype=b)})
        refuses(name, pa.rope, rope_args(), **{name: torch.zeros((T, H, D), dtype=torch.float16)})
        refuses(name, pa.rope, rope_args(), **{name: torch.zeros((T, H * D), dtype=b)})
    refuses("strides", pa.rope, rope_args(), q=torch.zeros((T, D, H), dtype=b).transpose(1, 2))
    refuses("strides", pa.rope, rope_args(), q=torch.zeros((H, T, D), dtype=b).transpose(0, 1))
    refuses("heads", pa.rope, rope_args(), k_out=torch.zeros((T, G + 1, D), dtype=b))
    refuses("heads", pa.rope, rope_args(), q_out=torch.zeros((T, H + 1, D), dtype=b))
    refuses("cos_sin", pa.rope, rope_args(), cos_sin=torch.zeros((9, D), dtype=torch.float64))
    refuses("cos_sin", pa.rope, rope_args(), cos_sin=torch.zeros(9 * D))
    for p in (torch.zeros(T), torch.zeros(T + 1, dtype=torch.int32),
              torch.zeros((T, 2), dtype=torch.int32), torch.zeros(T, dtype=torch.int64)):
        refuses("positions", pa.rope, rope_args(), positions=p)
    refuses("freq_axis", pa.rope, rope_args(), positions=torch.zeros((2, T), dtype=torch.int32),
            freq_axis=torch.zeros(D, dtype=torch.uint8))
    refuses("both or neither", pa.rope, rope_args(), k=None)
    refuses("both or neither", pa.rope, rope_args(), k_out=None)
    refuses("current device", pa.rope, rope_args())     # host tensors


def test_binding_of_rope_append():
    b = torch.bfloat16
    refuses("key", pa.rope_append_kv, append_args(), key=torch.zeros((T, G + 1, D), dtype=b),
            value=torch.zeros((T, G + 1, D), dtype=b))
    refuses("heads|value", pa.rope_append_kv, append_args(),
            value=torch.zeros((T, G - 1, D), dtype=b))
    refuses("key_out", pa.rope_append_kv, append_args(),
            key_out=torch.zeros((T, G, D), dtype=torch.float16))
    refuses("slot_mapping", pa.rope_append_kv, append_args(),
            slot_mapping=torch.zeros(T, dtype=torch.int32))
    refuses("both or neither", pa.rope_append_kv, append_args(), q=None)
    refuses("v_cache", pa.rope_append_kv, append_args(),
            v_cache=torch.zeros((NB - 1, G, 16, D), dtype=b))
    refuses("num_blocks", pa.rope_append_kv, append_args(), num_blocks=NB + 1)
    refuses("k_scale", pa.rope_append_kv, append_args(),
            k_cache=torch.zeros((NB, G, 16, D), dtype=torch.int8),
            v_cache=torch.zeros((NB, G, 16, D), dtype=torch.int8), k_scale=torch.zeros(3))
    refuses("current device", pa.rope_append_kv, append_args())


def test_plain_rotation():
    """Closed forms: position 0 changes nothing, a quarter turn swaps a pair, lengths stay,
    and scores of rotated rows depend on the distance of their positions alone."""
    rng = np.random.default_rng(0)
    tab = ref.table(64, 16)
    x = rng.standard_normal((5, 2, 32))
    for il in (False, True):
        pos = np.array([[0, 1, 2, 40, 63]])
        c, s = ref.angles(tab.astype(np.float64), pos)
        y = ref.rotate(x, c, s, il)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-6)
        back = ref.rotate(y, c, -s, il)
        assert np.allclose(back, x, atol=1e-6)
        q = np.zeros((1, 1, 16))
        q[0, 0, 0] = 1.0
        turned = ref.rotate(q, np.zeros((1, 8)), np.ones((1, 8)), il)
        assert turned[0, 0, 1 if il else 8] == 1.0 and turned[0, 0, 0] == 0.0
        a, b = x[:1], x[1:2]

        def score(m, n):
            cm, sm = ref.angles(tab, np.array([[m]]))
            cn, sn = ref.angles(tab, np.array([[n]]))
            return float((ref.rotate(a, cm, sm, il) * ref.rotate(b, cn, sn, il)).sum())

        assert abs(score(7, 3) - score(44, 40)) < 1e-5 * 64
    # frequency f takes the position of its axis
    c, _ = ref.angles(tab, np.array([[3], [5]]), [0, 1, 0, 1, 0, 1, 0, 1])
    assert c[0, 0] == tab[3, 0] and c[0, 1] == tab[5, 1] and c[0, 2] == tab[3, 2]


def test_plain_int8_is_the_oracles():
    import oracle
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 64)) * np.exp2(rng.integers(-20, 20, (40, 1)))).astype(np.float32)
    x[0] = 0
    x[1] = np.abs(x[1])
    x[2] = -np.abs(x[2])
    code, scale, zp = ref.quantise_int8(x)
    for i in range(len(x)):
        c, s, z = oracle.quantize_row(x[i])
        assert np.array_equal(c, code[i]) and s == scale[i] and z == zp[i]


def test_table_of_angles():
    from paged_kv_cache_154_gb300.engine import rope_table
    tab = rope_table(50, 16, device="cpu").numpy()
    assert tab.shape == (50, 16) and np.abs(tab - ref.table(50, 16)).max() < 1e-7
    # far positions: angles in 64 bits
    tab = rope_table(1 << 17, 8, device="cpu").numpy()
    p = (1 << 17) - 1
    want = np.cos(np.float64(p) * 10000.0 ** (-2 * np.arange(4) / 8))
    assert np.abs(tab[p, :4] - want).max() < 2.0 ** -24
    tab = rope_table(5, 4, inv_freq=[1.0, 0.5], factor=2.0, device="cpu").numpy()
    assert np.allclose(tab[3], [2 * np.cos(3), 2 * np.cos(1.5), 2 * np.sin(3), 2 * np.sin(1.5)])
    with pytest.raises(ValueError, match="inv_freq"):
        rope_table(5, 4, inv_freq=[1.0], device="cpu")


def test_engine_refuses_what_is_no_whole_prompt():
    from types import SimpleNamespace as Op
    from paged_kv_cache_154_gb300.engine import PagedKVCache
    cache = PagedKVCache(8, 1, 64, "f16", device="cpu")
    names = {}
    cache.reserve([Op(seq="a"), Op(seq="b")], names)
    cache.pool.seq_append_slots(names["b"], 3)
    x = torch.zeros((2, 1, 64), dtype=torch.float16)
    q = torch.zeros((4, 2, 64), dtype=torch.float16)

    def op(s):
        return Op(seq=s, k=x, v=x)

    with pytest.raises(ValueError, match="'b' holds 3 tokens"):
        cache.prepare_step([op("a"), op("b")], names, q, prompt=True)
    with pytest.raises(ValueError, match="twice"):
        cache.prepare_step([op("a"), op("a")], names, q, prompt=True)
    for bad in (dict(out_dtype=torch.float32), dict(partition_size=64), dict(shared_prefix=True)):
        with pytest.raises(ValueError, match="type of q"):
            cache.prepare_step([op("a")], names, q[:2], prompt=True, **bad)
    assert cache.pool.seq_len(names["a"]) == 0          # refused before anything is reserved
    si = cache.prepare_step([op("a")], names, q[:2], prompt=True)
    assert si.out.dtype == torch.float16 and si.workspace is None
    si = cache.prepare_step([op("b")], names, q[:2])
    assert si.out.dtype == torch.float32 and si.prompt_start is None
