"""Attention over packed prompts on the GPU against a plain 64-bit form.

Tolerance, derived before the first run. A score accumulates d exact products of 16-bit
numbers in fp32: off by at most (d + 4) 2^-24 sum |q k| scale, which the inputs keep under
2^-17 * 32 = 2.5e-4 (sum |q k| scale under 32 for d <= 128), so a weight is off by that much
relative to itself, and by 2^-21 from the exponential and the sums. A weight is rounded to
the 16-bit type once, half a step: 2^-8 (bf16, eps / 2) or 2^-11 (fp16) relative, and fp16
weights below 2^-14 by 2^-25 absolutely (n of them, their sum at least the 1 of the weight
that set the maximum). Each acts on sum p |v|; the result is off by half a step of its own."""
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


def make(seed, T, H, G, d, dtype, fused):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H + 2 * G, d), generator=gen)
    x[:, :H + G] *= 0.7     # sum |q k| scale about 0.31 sqrt(d) < 4 on average
    x = x.to(dtype).cuda()
    parts = x[:, :H], x[:, H:H + G], x[:, H + G:]
    return parts if fused else tuple(t.contiguous() for t in parts)


def starts(lens, behind=0):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()


def check(out, q, k, v, lens, scale, dtype):
    n = int(np.sum(lens))
    qh, kh, vh = host(q)[:n], host(k)[:n], host(v)[:n]
    want = ref.prompt_attention(qh, kh, vh, lens, scale)
    size = ref.prompt_attention(qh, kh, np.abs(vh), lens, scale)
    eps = torch.finfo(dtype).eps / 2
    tol = (eps + 2.5e-4 + 2.0 ** -21) * size * (1 + eps) + eps * np.abs(want) + 2.0 ** -24
    if dtype == torch.float16:
        tol += 2.0 ** -25 * max(lens) * np.abs(vh).max()
    got = host(out)[:n].astype(np.float64)
    off = np.abs(got - want) / tol
    assert np.isfinite(got).all() and off.max() <= 1, (off.max(), np.unravel_index(off.argmax(),
                                                                                   off.shape))


LENS = {
    "one": [1], "ones": [1, 1, 1, 1, 1], "short": [17, 33, 64, 100], "empty": [0, 5, 0, 0, 31, 0],
    "edges": [127, 128, 129, 255, 256, 257], "tails": [113, 112, 111, 97, 96, 95, 16, 15],
    "ragged": [1, 700, 3, 512, 40, 0, 1025],
    "long": [2049],
}


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("heads", [(8, 2, 64, "f16", False), (8, 2, 128, "bf16", True),
                                   (3, 3, 128, "f16", True), (7, 1, 64, "bf16", True),
                                   (28, 4, 128, "bf16", False)], ids=str)
def test_prompts(lens, heads):
    H, G, d, dt, fused = heads
    lens, dtype = LENS[lens], DT[dt]
    T = sum(lens) + 3                          # rows behind the last prompt
    q, k, v = make(len(lens), T, H, G, d, dtype, fused)
    k[T - 3:], v[T - 3:] = float("nan"), float("inf")
    out = torch.full((T, H + 1, d), 7.0, dtype=dtype, device="cuda")[:, :H]
    pa.prompt_attention(out, q, k, v, starts(lens), max(lens), d ** -0.5)
    assert pa.device_error() == 0
    check(out, q, k, v, lens, d ** -0.5, dtype)
    assert (out[T - 3:] == 7).all()


@pytest.mark.parametrize("group", [1, 5, 16, 43, 71, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_groups(group, d):
    lens = [130, 1, 61]
    q, k, v = make(group, sum(lens), group, 1, d, torch.float16, True)
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    pa.prompt_attention(out, q, k, v, starts(lens), 200, d ** -0.5)
    assert pa.device_error() == 0
    check(out, q, k, v, lens, d ** -0.5, torch.float16)


def test_values_of_other_prompts_do_not_matter():
    """NaN and infinities in the rows of one prompt leave every other prompt's as they were,
    bit for bit, wherever its tiles end."""
    lens = [33, 70, 129, 5, 250, 16, 1]
    for d in (64, 128):
        q, k, v = make(3, sum(lens), 4, 2, d, torch.bfloat16, False)
        s = starts(lens)
        a, b = torch.empty_like(q), torch.empty_like(q)
        pa.prompt_attention(a, q, k, v, s, max(lens), d ** -0.5)
        at = np.concatenate([[0], np.cumsum(lens)])
        for bad in (1, 3, 5):
            k2, v2, q2 = k.clone(), v.clone(), q.clone()
            rows = slice(int(at[bad]), int(at[bad + 1]))
            v2[rows], k2[rows] = float("nan"), float("inf")
            q2[rows] = float("-inf")
            pa.prompt_attention(b, q2, k2, v2, s, max(lens), d ** -0.5)
            keep = [i for i in range(sum(lens)) if not rows.start <= i < rows.stop]
            assert torch.equal(a[keep], b[keep])
            assert b[rows].isnan().all()


def test_growing_scores():
    """Scores that rise from tile to tile, so that the running maximum moves and O is scaled
    many times, and scores that fall, where later tiles add next to nothing."""
    T, d = 1400, 128
    q, k, v = make(5, T, 2, 1, d, torch.bfloat16, False)
    for sign in (1.0, -1.0):
        ramp = torch.linspace(0, 60, T, device="cuda")[:, None, None] * sign
        k2, q2 = k.clone() * 0.2, q.clone() * 0.2
        k2[..., :1] = ramp.to(k.dtype)
        q2[..., :1] = 8.0
        out = torch.empty_like(q)
        pa.prompt_attention(out, q2, k2, v, starts([T]), T, d ** -0.5)
        assert pa.device_error() == 0
        # scores up to 8 * 60 / 11.3 = 42.4 and an error of up to 3.4e-4 of a weight: within
        # the tolerance, whose first term alone is 2^-8
        check(out, q2, k2, v, [T], d ** -0.5, torch.bfloat16)


def test_scores_of_zero_and_scale_of_zero():
    T, d = 300, 64
    q, k, v = make(6, T, 2, 2, d, torch.float16, False)
    mean = torch.cumsum(v.double(), 0) / torch.arange(1, T + 1, device="cuda")[:, None, None]
    for q2, scale in ((torch.zeros_like(q), 1.0), (q, 0.0)):
        out = torch.empty_like(q)
        pa.prompt_attention(out, q2, k, v, starts([T]), T, scale)
        # weights of 1 are exact: fp32 sums of T values, and one rounding
        tol = 2.0 ** -11 * mean.abs() + T * 2.0 ** -23 * v.abs().max() + 2.0 ** -25
        assert ((out.double() - mean).abs() <= tol).all()


def test_cut_starts_and_lengths():
    """Starts outside the tensors and lengths past max_seq_len are cut, nothing else is
    written."""
    T, d = 64, 64
    q, k, v = make(8, T, 2, 1, d, torch.float16, False)
    out = torch.full_like(q, 3.0)
    s = torch.tensor([-5, 20, 18, 40, 1 << 30], dtype=torch.int32, device="cuda")
    pa.prompt_attention(out, q, k, v, s, 16, d ** -0.5)
    assert pa.device_error() == 0
    want = torch.full_like(q, 3.0)
    for a, n in ((0, 16), (18, 16), (40, 16)):     # the second of four is empty
        pa.prompt_attention(want[a:a + n], q[a:a + n], k[a:a + n], v[a:a + n], starts([n]), n,
                            d ** -0.5)
    assert torch.equal(out, want)


def test_many_prompts():
    """More prompts than one launch takes, among them empty ones."""
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 9, 1300).tolist()
    q, k, v = make(10, sum(lens), 2, 1, 64, torch.bfloat16, True)
    out = torch.empty((sum(lens), 2, 64), dtype=torch.bfloat16, device="cuda")
    pa.prompt_attention(out, q, k, v, starts(lens), 8, 0.125)
    assert pa.device_error() == 0
    check(out, q, k, v, lens, 0.125, torch.bfloat16)


def test_rows_far_apart():
    """Offsets past 2^32 bytes and 2^31 elements, in every tensor."""
    lens, d = [3, 2], 128
    near = make(11, 5, 4, 2, d, torch.bfloat16, False)
    want = torch.empty((5, 4, d), dtype=torch.bfloat16, device="cuda")
    pa.prompt_attention(want, *near, starts(lens), 3, d ** -0.5)
    store = torch.zeros(4 * (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    far = []
    at = 0
    for t in (want, *near):
        x = store[at:].as_strided((5, t.shape[1], d), (1 << 30, d, 1), at)
        far.append(x)
        at += t.shape[1] * d
    for x, t in zip(far[1:], near):
        x.copy_(t)
    pa.prompt_attention(*far, starts(lens), 3, d ** -0.5)
    assert torch.equal(far[0], want)


def test_repeated_runs_are_equal():
    lens = [900, 31, 1500, 7]
    q, k, v = make(12, sum(lens), 8, 2, 128, torch.bfloat16, True)
    outs = [torch.empty((sum(lens), 8, 128), dtype=torch.bfloat16, device="cuda")
            for _ in range(4)]
    for o in outs:
        pa.prompt_attention(o, q, k, v, starts(lens), 1500, 0.09)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_streams_and_graphs():
    lens = [300, 20, 129]
    q, k, v = make(13, sum(lens), 4, 1, 64, torch.float16, True)
    s = starts(lens)
    outs = [torch.empty((sum(lens), 4, 64), dtype=torch.float16, device="cuda") for _ in range(3)]

    def call(o, stream=None):
        pa.prompt_attention(o, q, k, v, s, 300, 0.125, stream=stream)

    call(outs[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(outs[1], side)          # and at the same time on the current one
    call(outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[2])
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        q.mul_(0.5)
        s[1] -= 7                 # other prompts in the same buffers
        call(outs[0])
        call(outs[1])
        torch.cuda.synchronize()


def test_validation_names_the_prompt(monkeypatch):
    q, k, v = make(14, 10, 2, 1, 64, torch.float16, False)
    monkeypatch.setenv("PA_VALIDATE", "1")
    for s in ([0, 4, 3], [0, 11, 11], [-1, 4, 5], [0, 9, 10]):
        with pytest.raises(pa.PAError, match="prompt [01] has tokens"):
            pa.prompt_attention(torch.empty_like(q), q, k, v,
                                torch.tensor(s, dtype=torch.int32, device="cuda"), 8, 0.1)
    pa.prompt_attention(torch.empty_like(q), q, k, v, starts([4, 6]), 8, 0.1)
    assert pa.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_sums_of_long_prompts(d):
    """With a workspace the weighted sums of values of one sign stay as near to the 64-bit
    ones over 131072 keys as over a few; the workspace holds NaN before, serves calls of other
    lengths, and a part for 7 CTAs serves too. Tolerance: a span of 8192 keys is 512 sums of
    16, each cut off by a step of 24 bits at most, 2^-23 of what is there so far: 512 * 2^-23 =
    6.1e-5 of a span's sum. The mean over d columns also holds the rounding of the outputs,
    which lie around 1: 2^-10 / sqrt(12 * 64) a standard deviation of it, 4 of them 1.4e-4."""
    T, H = 131072, 2
    gen = torch.Generator(device="cuda").manual_seed(d)
    q, k = ((torch.randn((T, n, d), device="cuda", generator=gen) * 0.3).half() for n in (H, 1))
    v = (torch.rand((T, 1, d), device="cuda", generator=gen) + 0.5).half()
    n = pa.prompt_attention_workspace_size(d, T)
    start = torch.tensor([0, 5000, T], dtype=torch.int32, device="cuda")
    outs = []
    for size in (n, 7 * n // 152):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        for _ in range(2):
            pa.prompt_attention(out, q, k, v, start, T, d ** -0.5, ws)
        outs.append(out)
    assert pa.device_error() == 0
    assert torch.equal(*outs)
    short = torch.empty_like(q[:5000])
    pa.prompt_attention(short, q[:5000], k[:5000], v[:5000], start[:2], 5000, d ** -0.5)
    assert torch.equal(outs[0][:5000], short)
    for row in (5000 + 8191, 5000 + 8192, 90000, T - 1):
        s = (q[row].double() @ k[5000:row + 1, 0].double().t()) * d ** -0.5
        want = torch.softmax(s, -1) @ v[5000:row + 1, 0].double()
        off = (outs[0][row].double() - want) / want
        # an output: its rounding, and at most as much of every weight's
        assert off.abs().max() < 2.0 ** -10 + 6.1e-5
        assert abs(off.mean().item()) < 6.1e-5 + 1.4e-4


@pytest.mark.parametrize("d", [64, 128])
def test_kept_sums_follow_the_maximum(d):
    """Scores that rise over several spans, so that the sums of earlier ones are scaled, and
    that fall, so that they outweigh the later ones."""
    T = 20000
    q, k, v = make(15, T, 2, 1, d, torch.bfloat16, False)
    ws = torch.full((pa.prompt_attention_workspace_size(d, T),), 255, dtype=torch.uint8,
                    device="cuda")
    for sign in (1.0, -1.0):
        k2, q2 = k.clone() * 0.2, q.clone() * 0.2
        k2[..., :1] = (torch.linspace(0, 40, T, device="cuda")[:, None, None] * sign).to(k.dtype)
        q2[..., :1] = 0.6 * d ** 0.5
        out = torch.empty_like(q)
        pa.prompt_attention(out, q2, k2, v, starts([T]), T, d ** -0.5, ws)
        assert pa.device_error() == 0
        eps = torch.finfo(torch.bfloat16).eps / 2
        for row in (8191, 8192, 8193, 13000, 16384, T - 1):
            s = (q2[row].double() @ k2[:row + 1, 0].double().t()) * d ** -0.5
            w, x = torch.softmax(s, -1), v[:row + 1, 0].double()
            want, size = w @ x, w @ x.abs()
            # scores up to 24, sums of d terms and the power: 24 * 132 * 2^-24 = 1.9e-4 of a
            # weight; the sums of products 6.1e-5
            tol = (eps + 2.6e-4 + 2.0 ** -21) * size * (1 + eps) + eps * want.abs() + 2.0 ** -24
            assert ((out[row].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_weights_far_above_the_reference(d, dt):
    """Keys from 40 on score 14.7 binary orders above the first ones, by which the reference of
    the weights is taken: it does not move, and all weights are near 2^14.7 (fp16 ends at 2^16)."""
    T = 600
    q, k, v = make(17, T, 2, 1, d, DT[dt], False)
    k2, q2 = k * 0.2, q * 0.2
    k2[:40, :, 0], k2[40:, :, 0] = 0, 2
    q2[..., 0] = 5.1 * d ** 0.5
    out = torch.empty_like(q)
    pa.prompt_attention(out, q2, k2, v, starts([T]), T, d ** -0.5)
    assert pa.device_error() == 0
    check(out, q2, k2, v, [T], d ** -0.5, DT[dt])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("first", [70, 127, 128, 190])
def test_weights_far_above_the_reference_from_any_key(first, dt):
    """As above from other keys on: of a tile's second half, where the reference stays, of the
    next tile, where the sum of many moves it, and with a last tile of few keys."""
    T, d = 385, 64
    q, k, v = make(18, T, 3, 1, d, DT[dt], False)
    k2, q2 = k * 0.2, q * 0.2
    k2[:first, :, 0], k2[first:, :, 0] = 0, 2
    q2[..., 0] = 5.1 * d ** 0.5
    out = torch.empty_like(q)
    pa.prompt_attention(out, q2, k2, v, starts([T]), T, d ** -0.5)
    assert pa.device_error() == 0
    check(out, q2, k2, v, [T], d ** -0.5, DT[dt])
