"""Rotary positions on the GPU against plain forms: rows turned on their own and on the
way into a cache of every type, bit for bit against the same formula with every product
and sum rounded to fp32, and within the tolerance below of the 64-bit form.

Tolerance, derived before the first run: a' = a c - b s has two products and a sum, each
off by at most half a step (2^-24 relative), so by 2^-24 (2 |a c| + 2 |b s|) in all, and
the 16-bit result is off by half a step of its own, 2^-8 (bf16) or 2^-11 (fp16) of itself."""
import numpy as np
import pytest
import torch

import paged_kv_cache_154_gb300 as pa
from oracle import rotary as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def host(t):
    return t.float().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy().reshape(-1)


def rows(gen, T, H, G, d, dtype, fused):
    """q, k and v on the device; a fused projection's rows hold a margin besides."""
    def make(n, wide):
        x = torch.randn((T, n, d), generator=gen)
        x[..., ::7] *= 4
        return x.to(dtype).cuda()
    if fused:
        x = make(H + 2 * G + 1, True)
        return x[:, :H], x[:, H:H + G], x[:, H + G:H + 2 * G]
    return make(H, False), make(G, False), make(G, False)


def positions(rng, T, axes, most):
    return rng.integers(0, most, (axes, T)).astype(np.int32)


def axis_of(rng, axes, n):
    return None if axes == 1 else rng.integers(0, axes, n).astype(np.uint8)


def on_gpu(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def within(got, x, c, s, il, dtype):
    """The 64-bit form and the tolerance of this file's head."""
    want = ref.rotate(x, c, s, il)
    n = c.shape[1]
    size = np.abs(x).astype(np.float64)
    turned = ref.rotate(size, np.abs(c), -np.abs(s), il)   # |a c| + |b s| in the first halves
    other = ref.rotate(size, np.abs(c), np.abs(s), il)     # |b c| + |a s| in the second
    first = np.zeros(x.shape[-1], bool)
    first[(np.arange(n) * 2) if il else np.arange(n)] = True
    bound = np.where(first, np.abs(turned), np.abs(other))
    eps = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133   # half a subnormal step
    tol = 2.0 ** -23 * bound * (1 + eps) + eps * np.abs(want) + tiny
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


SHAPES = [  # T, H, G, d, rd, interleaved, axes, dtype, fused
    (1, 8, 2, 128, 128, False, 1, "bf16", False),
    (1, 1, 1, 64, 64, True, 1, "f16", True),
    (3, 5, 0, 64, 32, False, 1, "bf16", False),
    (33, 32, 8, 128, 128, False, 1, "bf16", True),
    (17, 28, 4, 128, 96, False, 3, "f16", True),
    (64, 3, 3, 64, 16, True, 2, "bf16", True),
    (5, 7, 1, 128, 48, True, 4, "f16", False),
    (7, 71, 1, 64, 64, False, 3, "bf16", False),
    (1025, 2, 1, 128, 64, False, 1, "f16", True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(shape, inverse):
    T, H, G, d, rd, il, axes, dt, fused = shape
    gen = torch.Generator().manual_seed(T + H)
    rng = np.random.default_rng(T)
    dtype, most = DT[dt], 5000
    q, k, _ = rows(gen, T, H, max(G, 1), d, dtype, fused)
    tab = ref.table(most, rd)
    pos, axis = positions(rng, T, axes, most), axis_of(rng, axes, rd // 2)
    c, s = ref.angles(tab, pos, axis)
    if inverse:
        s = -s
    before = q.clone(), k.clone()
    room = torch.full((T, H + 3, d), 7.0, dtype=dtype, device="cuda")
    qo, ko = room[:, 1:H + 1], torch.full_like(k, 7.0, memory_format=torch.contiguous_format)
    pos_d = on_gpu(pos[0] if axes == 1 else pos)
    pa.rope(qo, q, ko if G else None, k if G else None, on_gpu(tab), pos_d, il, on_gpu(axis),
            inverse)
    assert pa.device_error() == 0
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    assert (room[:, 0] == 7).all() and (room[:, H + 1:] == 7).all()
    for got, x in ((qo, q),) + (((ko, k),) if G else ()):
        step = torch.from_numpy(ref.rotate(host(x), c, s, il, np.float32)).to(dtype)
        assert np.array_equal(bits(got), bits(step))
        within(host(got).astype(np.float64), host(x), c, s, il, dtype)
    if G == 0:
        assert (ko == 7).all()


def test_rope_in_place():
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((50, 12, 64), generator=gen).to(torch.bfloat16).cuda()
    tab = on_gpu(ref.table(100, 64))
    pos = torch.arange(50, dtype=torch.int32).cuda()
    want_q, want_k = torch.empty_like(x[:, :8]), torch.empty_like(x[:, 8:10])
    pa.rope(want_q, x[:, :8], want_k, x[:, 8:10], tab, pos)
    rest = x[:, 10:].clone()
    pa.rope(x[:, :8], x[:, :8], x[:, 8:10], x[:, 8:10], tab, pos)
    assert torch.equal(x[:, :8], want_q) and torch.equal(x[:, 8:10], want_k)
    assert torch.equal(x[:, 10:], rest)


def test_gradient_is_the_inverse():
    """<w, rope(x)> is linear in x: its gradient is rope(w) turned the other way, against the
    formula's transpose and against differences. Values are small integers and the table's
    entries multiples of 2^-5, so every product and sum is exact in fp32, and in fp16."""
    rng = np.random.default_rng(5)
    T, H, d, rd = 6, 3, 64, 32
    tab = (rng.integers(-16, 17, (20, rd)) / 32).astype(np.float32)
    pos = rng.integers(0, 20, T).astype(np.int32)
    x = rng.integers(-8, 9, (T, H, d)).astype(np.float32)
    w = rng.integers(-8, 9, (T, H, d)).astype(np.float32)

    def run(a, inverse):
        t = torch.from_numpy(a).to(torch.float16).cuda()
        out = torch.empty_like(t)
        pa.rope(out, t, None, None, on_gpu(tab), on_gpu(pos), inverse=inverse)
        return host(out).astype(np.float64)

    grad = run(w, True)
    assert (w * run(x, False)).sum() == (grad * x).sum()
    for i in (0, 15, 16, 31, 32, 63):       # one step of one element
        e = x.copy()
        e[2, 1, i] += 1
        assert (w * run(e, False)).sum() - (w * run(x, False)).sum() == grad[2, 1, i]


@pytest.mark.parametrize("axes", [1, 3])
def test_a_position_outside_the_table_leaves_its_token(axes):
    T, most = 40, 16
    x = torch.ones((T, 5, 64), dtype=torch.float16, device="cuda")
    pos = np.arange(axes * T).reshape(axes, T).astype(np.int32) % most
    pos[-1, 3], pos[0, 7], pos[0, 39] = most, -1, 1 << 30
    out = torch.full_like(x, 9.0)
    axis = None if axes == 1 else torch.zeros(32, dtype=torch.uint8, device="cuda")
    tab = on_gpu(ref.table(most, 64))
    pa.rope(out, x, None, None, tab, on_gpu(pos), freq_axis=axis)
    assert pa.device_error() == pa.DEVERR_BAD_SLOT
    left = (out == 9).all(2).all(1)
    assert left.nonzero().flatten().tolist() == [3, 7, 39]
    if axes > 1:
        out.fill_(9.0)
        axis[5] = axes
        pa.rope(out, x, None, None, tab, on_gpu(pos), freq_axis=axis)
        assert pa.device_error() == pa.DEVERR_BAD_SLOT and (out == 9).all()


def make_cache(kind, nb, G, d, dtype, rng):
    """Cache arrays full of one byte, so that every slot not written shows."""
    width = d // 2 if kind == "int4" else d
    t = {"int8": torch.int8, "int4": torch.uint8, "fp8": torch.float8_e4m3fn}.get(kind, dtype)
    c = {}
    for n in ("k", "v"):
        size = nb * G * 16 * width * (2 if t == dtype else 1)
        c[n + "_cache"] = torch.full((size,), 0x3c, dtype=torch.uint8,
                                     device="cuda").view(t).view(nb, G, 16, width)
        c[n + "_scale"] = c[n + "_zp"] = None
        if kind in ("int8", "int4"):
            row = (nb, G, 16) + ((d // 64,) if kind == "int4" else ())
            c[n + "_scale"] = torch.full(row, 77.0, device="cuda")
            c[n + "_zp"] = torch.full(row, 99, dtype=torch.int8, device="cuda")
        if kind == "fp8":
            c[n + "_scale"] = on_gpu((rng.random(G) * 0.1 + 0.02).astype(np.float32))
    return c


def expected(kind, cache, slots, x, n, dtype):
    """The cache arrays after fp32 rows x [T, G, d] went to their slots."""
    ok = slots >= 0
    b, o = slots[ok] // 16, slots[ok] % 16
    x = x[ok]
    code = bits(cache[n + "_cache"]).reshape(*cache[n + "_cache"].shape[:3], -1).copy()
    if kind in ("int8", "int4"):
        got, scale, zp = ref.quantise(x, kind)
        code[b, :, o] = got.view(np.uint8)
        sc, z = (cache[n + e].cpu().numpy().copy() for e in ("_scale", "_zp"))
        sc[b, :, o], z[b, :, o] = scale, zp
        return code, sc, z
    if kind == "fp8":
        y = x / cache[n + "_scale"].cpu().numpy()[:, None]
        y = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn)
        code[b, :, o] = y.view(torch.uint8).numpy()
    else:
        y = torch.from_numpy(x).to(dtype)
        code[b, :, o] = y.view(torch.uint8).numpy().reshape(*x.shape[:2], -1)
    return code, None, None


def check_cache(kind, cache, want):
    for n in ("k", "v"):
        code, scale, zp = want[n]
        assert np.array_equal(bits(cache[n + "_cache"]), code.reshape(-1)), n
        if scale is not None:
            assert np.array_equal(cache[n + "_scale"].cpu().numpy(), scale), n
            assert np.array_equal(cache[n + "_zp"].cpu().numpy(), zp), n


def scattered(rng, T, nb, skipped):
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    slots[rng.permutation(T)[:skipped]] = -1 - rng.integers(0, 1 << 40, skipped)
    return slots


@pytest.mark.parametrize("kind", ["same", "int8", "fp8", "int4"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[2]], ids=str)
def test_rope_append(kind, shape):
    T, H, G, d, rd, il, axes, dt, fused = shape
    gen = torch.Generator().manual_seed(2 * T + H)
    rng = np.random.default_rng(T + 1)
    dtype, most = DT[dt], 5000
    kind = dt if kind == "same" else kind
    q, k, v = rows(gen, T, H, G, d, dtype, fused)
    tab = ref.table(most, rd)
    pos, axis = positions(rng, T, axes, most), axis_of(rng, axes, rd // 2)
    c, s = ref.angles(tab, pos, axis)
    nb = T // 16 + 5
    slots = scattered(rng, T, nb, T // 7)
    cache = make_cache(kind, nb, G, d, dtype, rng)
    kr = ref.rotate(host(k), c, s, il, np.float32)
    want = {"k": expected(kind, cache, slots, kr, "k", dtype),
            "v": expected(kind, cache, slots, host(v), "v", dtype)}
    qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty((T, G, d),
                                                                                   dtype=dtype,
                                                                                   device="cuda")
    pa.rope_append_kv(qo, q, k, v, cache["k_cache"], cache["v_cache"], on_gpu(slots), on_gpu(tab),
                      on_gpu(pos[0] if axes == 1 else pos), None, cache["k_scale"],
                      cache["v_scale"], cache["k_zp"], cache["v_zp"], ko, il, on_gpu(axis))
    assert pa.device_error() == 0
    check_cache(kind, cache, want)
    step = torch.from_numpy(ref.rotate(host(q), c, s, il, np.float32)).to(dtype)
    assert np.array_equal(bits(qo), bits(step))
    assert np.array_equal(bits(ko), bits(torch.from_numpy(kr).to(dtype)))
    # without queries, without rows of keys; values as pa_append_kv has them
    again = make_cache(kind, nb, G, d, dtype, rng)
    for n in ("k_scale", "v_scale"):
        if kind == "fp8":
            again[n] = cache[n]
    pa.rope_append_kv(None, None, k, v, again["k_cache"], again["v_cache"], on_gpu(slots),
                      on_gpu(tab), on_gpu(pos[0] if axes == 1 else pos), nb, again["k_scale"],
                      again["v_scale"], again["k_zp"], again["v_zp"], None, il, on_gpu(axis))
    check_cache(kind, again, want)
    plain = make_cache(kind, nb, G, d, dtype, rng)
    for n in ("k_scale", "v_scale"):
        if kind == "fp8":
            plain[n] = cache[n]
    pa.append_kv(k.contiguous(), v.contiguous(), plain["k_cache"], plain["v_cache"], on_gpu(slots),
                 nb, plain["k_scale"], plain["v_scale"], plain["k_zp"], plain["v_zp"])
    assert np.array_equal(bits(plain["v_cache"]), bits(cache["v_cache"]))


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_ranges_of_quantised_rows(kind):
    """Rows of zeros, of one sign, of one value, and from the smallest to the largest fp32
    numbers that bf16 holds (their range finite): codes, scales and zero points bit for bit."""
    rng = np.random.default_rng(11)
    T, G, d, rd = 96, 2, 128, 128
    x = rng.standard_normal((T, G, d)).astype(np.float32)
    x *= np.exp2(np.linspace(-130, 125, T)).astype(np.float32)[:, None, None]
    x[0], x[1], x[2] = 0, np.abs(x[60]), -np.abs(x[61])
    x[3], x[4] = 2.5, -2.5
    x[5] = np.float32(2.0 ** -133)
    x[6, :, 1:] = 0
    k = torch.from_numpy(np.clip(x, -2.0 ** 125, 2.0 ** 125)).to(torch.bfloat16).cuda()
    v = k.flip(0).contiguous()
    tab = ref.table(300, rd)
    pos = rng.integers(0, 300, (1, T)).astype(np.int32)
    c, s = ref.angles(tab, pos)
    slots = scattered(rng, T, 8, 3)
    cache = make_cache(kind, 8, G, d, torch.bfloat16, rng)
    with np.errstate(under="ignore"):
        want = {"k": expected(kind, cache, slots, ref.rotate(host(k), c, s, False, np.float32),
                              "k", torch.bfloat16),
                "v": expected(kind, cache, slots, host(v), "v", torch.bfloat16)}
    pa.rope_append_kv(None, None, k, v, cache["k_cache"], cache["v_cache"], on_gpu(slots),
                      on_gpu(tab), on_gpu(pos[0]), None, cache["k_scale"], cache["v_scale"],
                      cache["k_zp"], cache["v_zp"])
    check_cache(kind, cache, want)


def test_bad_slots_and_positions_on_the_way_in():
    """A slot outside the pool keeps the cache as it was and still gives the rows; a position
    outside the table leaves the token whole."""
    rng = np.random.default_rng(13)
    T, G, d, nb = 20, 2, 64, 4
    x = torch.randn((T, 3 * G, d), generator=torch.Generator().manual_seed(1)).half().cuda()
    tab = on_gpu(ref.table(32, d))
    pos = np.arange(T).astype(np.int32)
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    good = slots.copy()
    slots[4], slots[5] = nb * 16, 1 << 50
    pos[9] = 32
    cache, want = make_cache("f16", nb, G, d, torch.float16, rng), make_cache(
        "f16", nb, G, d, torch.float16, rng)
    qo, ko = torch.full_like(x[:, :G], 5.0), torch.full_like(x[:, :G], 5.0)
    pa.rope_append_kv(qo, x[:, :G], x[:, G:2 * G], x[:, 2 * G:], cache["k_cache"],
                      cache["v_cache"], on_gpu(slots), tab, on_gpu(pos), key_out=ko)
    assert pa.device_error() == pa.DEVERR_BAD_SLOT
    keep = [i for i in range(T) if i not in (4, 5, 9)]
    rot = torch.empty_like(x[:, :2 * G])
    pos[9] = 0
    pa.rope(rot, x[:, :2 * G], None, None, tab, on_gpu(pos))
    pa.append_kv(rot[keep, G:].contiguous(), x[keep, 2 * G:].contiguous(), want["k_cache"],
                 want["v_cache"], on_gpu(good[keep]))
    assert torch.equal(cache["k_cache"], want["k_cache"])
    assert torch.equal(cache["v_cache"], want["v_cache"])
    rows_ = [i for i in range(T) if i != 9]
    assert torch.equal(qo[rows_], rot[rows_, :G]) and torch.equal(ko[rows_], rot[rows_, G:])
    assert (qo[9] == 5).all() and (ko[9] == 5).all()


def test_validation_names_the_entry(monkeypatch):
    monkeypatch.setenv("PA_VALIDATE", "1")
    x = torch.ones((4, 2, 64), dtype=torch.float16, device="cuda")
    tab = on_gpu(ref.table(8, 64))
    with pytest.raises(pa.PAError, match="position 8 of token 2"):
        pa.rope(torch.empty_like(x), x, None, None, tab, on_gpu(np.array([0, 1, 8, 3], np.int32)))
    with pytest.raises(pa.PAError, match="frequency 31 has axis 2"):
        axis = np.zeros(32, np.uint8)
        axis[31] = 2
        pa.rope(torch.empty_like(x), x, None, None, tab, on_gpu(np.zeros((2, 4), np.int32)),
                freq_axis=on_gpu(axis))
    pa.rope(torch.empty_like(x), x, None, None, tab, on_gpu(np.zeros(4, np.int32)))
    assert pa.device_error() == 0


def test_tokens_far_apart():
    """Offsets past 2^32 bytes and 2^31 elements."""
    store = torch.zeros(3 * (1 << 30), dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((3, 4, 128), (1 << 30, 128, 1))
    x.copy_(torch.randn((3, 4, 128), generator=torch.Generator().manual_seed(7)))
    near = x.contiguous()
    tab = on_gpu(ref.table(8, 128))
    pos = torch.tensor([1, 3, 5], dtype=torch.int32, device="cuda")
    want = torch.empty_like(near)
    pa.rope(want, near, None, None, tab, pos)
    pa.rope(x[:, :2], x[:, :2], x[:, 2:], x[:, 2:], tab, pos)
    assert torch.equal(x, want)


def test_streams_and_graphs():
    """A call on another stream than the current one, and a captured call that is replayed
    on new inputs in the same buffers."""
    rng = np.random.default_rng(17)
    T, H, G, d, nb = 30, 4, 2, 128, 6
    x = torch.randn((T, H + 2 * G, d), generator=torch.Generator().manual_seed(2)).to(
        torch.bfloat16).cuda()
    tab = on_gpu(ref.table(64, d))
    pos = on_gpu(rng.integers(0, 64, T).astype(np.int32))
    slots = on_gpu(scattered(rng, T, nb, 2))

    def call(cache, qo, stream=None):
        pa.rope_append_kv(qo, x[:, :H], x[:, H:H + G], x[:, H + G:], cache["k_cache"],
                          cache["v_cache"], slots, tab, pos, None, cache["k_scale"],
                          cache["v_scale"], cache["k_zp"], cache["v_zp"], stream=stream)

    caches = [make_cache("int8", nb, G, d, torch.bfloat16, rng) for _ in range(3)]
    outs = [torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    call(caches[0], outs[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(caches[1], outs[1], side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(caches[2], outs[2])
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for i in (1, 2):
            assert torch.equal(outs[0], outs[i])
            for n in ("k_cache", "v_cache", "k_scale", "v_zp"):
                assert torch.equal(caches[0][n], caches[i][n])
        x.mul_(0.5)
        call(caches[0], outs[0])
        call(caches[1], outs[1])
        torch.cuda.synchronize()


def test_slots_far_into_a_cache():
    """Cache offsets past 2^32 bytes and 2^31 elements, in the first and the last blocks."""
    nb, G, d, T = 140000, 8, 128, 40
    gen = torch.Generator().manual_seed(21)
    k, v = (torch.randn((T, G, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    tab = on_gpu(ref.table(64, d))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.cat([torch.arange(20), nb * 16 - 20 + torch.arange(20)]).cuda()
    kc, vc = (torch.zeros((nb, G, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa.rope_append_kv(None, None, k, v, kc, vc, slots, tab, pos)
    rows_ = torch.empty_like(k), torch.empty_like(v)
    pa.gather_kv(*rows_, kc, vc, slots)
    assert pa.device_error() == 0
    want = torch.empty_like(k)
    pa.rope(want, k, None, None, tab, pos)
    assert torch.equal(rows_[0], want) and torch.equal(rows_[1], v)
    assert int(kc[2:-2].count_nonzero()) == 0 and int(vc[2:-2].count_nonzero()) == 0
