"""The way of a prompt or a step into the paged KV cache, as cases to be measured.

Three operators between a model's projection and the cache:

* "rope":   query and key rows rotated by their positions, of one axis (text) or of several
            (time, height and width of images and video) (rope);
* "append": the same for a step or prompt that enters the cache: queries rotated, keys rotated
            and written through the slot mapping, values written; an 8- or 4-bit cache is read
            back at the values that it holds (rope_append_kv, gather_kv);
* "prompt": causal attention over whole prompts, packed one after another, with grouped heads
            (prompt_attention).

Where `own` is false, `run` computes them with elementary torch operations in 32 bits; where it
is true, with the library's calls.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16     # tokens per cache block
GROUP = 64     # elements that share a 4-bit scale and zero point
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
SCORES = 1 << 31   # logits that the plain form of "prompt" holds at once


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the queries and keys of one decode step of 64 sequences at scattered positions
        {"name": "rope_step", "kind": "rope", "tokens": 64, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "rotary_dim": 128, "interleaved": False, "axes": 1, "sections": True,
         "inverse": False, "prompts": 0, "dtype": "bf16", "fused": True, "positions": 131072},
        # images and video: tokens on a grid, each frequency at the position of one of three axes
        {"name": "rope_image", "kind": "rope", "tokens": 8191, "heads": 28, "kv_heads": 4,
         "head_dim": 128, "rotary_dim": 128, "interleaved": False, "axes": 3, "sections": True,
         "inverse": False, "prompts": 1, "dtype": "bf16", "fused": True, "positions": 32768},
        # queries and keys turned back, pairs next to each other, a quarter of every head
        {"name": "rope_back", "kind": "rope", "tokens": 2047, "heads": 16, "kv_heads": 16,
         "head_dim": 64, "rotary_dim": 16, "interleaved": True, "axes": 1, "sections": True,
         "inverse": True, "prompts": 3, "dtype": "f16", "fused": False, "positions": 8192},
        # a step of 64 sequences enters a 16-bit cache, with two padded rows
        {"name": "append_step", "kind": "append", "tokens": 66, "padded": 2, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "rotary_dim": 128, "interleaved": False, "axes": 1,
         "sections": True, "prompts": 0, "cache": "bf16", "dtype": "bf16", "fused": True,
         "positions": 131072},
        # a step enters an 8-bit cache, its tokens on three axes
        {"name": "append_step_int8", "kind": "append", "tokens": 33, "padded": 0, "heads": 64,
         "kv_heads": 8, "head_dim": 128, "rotary_dim": 128, "interleaved": False, "axes": 3,
         "sections": False, "prompts": 0, "cache": "int8", "dtype": "bf16", "fused": True,
         "positions": 32768},
        # 8 prompts of 2048 tokens enter a 16-bit cache
        {"name": "append_prompts", "kind": "append", "tokens": 16384, "padded": 0, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "rotary_dim": 128, "interleaved": False, "axes": 1,
         "sections": True, "prompts": 8, "cache": "bf16", "dtype": "bf16", "fused": True,
         "positions": 131072},
        # prompts enter a 4-bit cache, half of every head rotated, pairs next to each other
        {"name": "append_prompts_int4", "kind": "append", "tokens": 6001, "padded": 0, "heads": 64,
         "kv_heads": 8, "head_dim": 128, "rotary_dim": 64, "interleaved": True, "axes": 1,
         "sections": True, "prompts": 3, "cache": "int4", "dtype": "f16", "fused": False,
         "positions": 8192},
        # four short prompts, the smallest call: latency
        {"name": "prompt_tiny", "kind": "prompt", "seqs": 4, "len_lo": 17, "len_hi": 100,
         "heads": 8, "kv_heads": 2, "head_dim": 64, "dtype": "f16", "fused": False, "lens_seed": 1},
        # a batch of prompts of very different lengths
        {"name": "prompt_batch", "kind": "prompt", "seqs": 16, "len_lo": 200, "len_hi": 2000,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "fused": True,
         "lens_seed": 2},
        # heads that share nothing, 64 wide
        {"name": "prompt_heads64", "kind": "prompt", "seqs": 6, "len_lo": 1000, "len_hi": 4096,
         "heads": 16, "kv_heads": 16, "head_dim": 64, "dtype": "f16", "fused": True,
         "lens_seed": 3},
        # groups of seven heads
        {"name": "prompt_groups7", "kind": "prompt", "seqs": 2, "len_lo": 4097, "len_hi": 5003,
         "heads": 28, "kv_heads": 4, "head_dim": 128, "dtype": "bf16", "fused": True,
         "lens_seed": 4},
        # one long prompt
        {"name": "prompt_long", "kind": "prompt", "seqs": 1, "len_lo": 32768, "len_hi": 32768,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "fused": True,
         "lens_seed": 5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "append", "prompt", "prompt", "prompt"])
    d = rng.choice([64, 128])
    c = {"kind": kind, "head_dim": d, "dtype": rng.choice(["bf16", "f16"]),
         "kv_heads": rng.choice([1, 2, 3, 4, 8]), "fused": rng.random() < 0.5}
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 7, 8])
    if kind == "prompt":
        c["lens_seed"] = rng.randrange(1 << 20)
        c["seqs"] = _log_int(rng, 1, 64)
        # the logits of all heads and of the padded batch, up to a part of the long prompt's
        most = math.isqrt((1 << 33) // (c["seqs"] * c["heads"]))
        c["len_hi"] = _log_int(rng, 1, min(32768, most))
        c["len_lo"] = max(1, int(c["len_hi"] * rng.choice([0.02, 0.3, 0.9])))
        return c
    c.update(rotary_dim=rng.choice([d, d, d // 2, 16 * rng.randrange(1, d // 16)]),
             interleaved=rng.random() < 0.4, axes=rng.choice([1, 1, 2, 3]),
             sections=rng.random() < 0.7, prompts=rng.choice([0, 1, 3, 8]),
             positions=rng.choice([8192, 32768, 131072]))
    c["tokens"] = _log_int(rng, max(1, c["prompts"]), 8192)
    if kind == "rope":
        c["inverse"] = rng.random() < 0.3
    else:
        c["cache"] = rng.choice([c["dtype"], c["dtype"], "int8", "fp8", "int4"])
        c["padded"] = rng.choice([0, 0, 1, 5]) if c["tokens"] > 8 else 0
    return c


def _lens(case):
    """Lengths of the prompts; the case alone decides them."""
    r = np.random.RandomState(case["lens_seed"])
    return r.randint(case["len_lo"], case["len_hi"] + 1, case["seqs"]).astype(np.int64)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows(shape, gen, dev, dtype):
    """Rows of a projection: normal, with a few channels of a larger range, as models have."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    x[..., ::29] *= 3.0
    return x.to(dtype)


def _projection(case, T, gen, dev):
    """q, k and v rows [T, heads, d]: parts of one row a token where the projection is fused."""
    H, G, d, dtype = case["heads"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    if case["fused"]:
        x = _rows((T, H + 2 * G, d), gen, dev, dtype)
        return x[:, :H], x[:, H:H + G], x[:, H + G:]
    return tuple(_rows((T, n, d), gen, dev, dtype) for n in (H, G, G))


def _table(rotary_dim, positions, dev):
    """cos and sin of position / 10000 ^ (2 f / rotary_dim), [positions, rotary_dim]."""
    f = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=dev) / rotary_dim
    angle = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** -f
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def _positions(case, gen, dev):
    """int32 [axes, tokens]: prompts one after another, or the scattered ones of a step."""
    T, A, P = case["tokens"], case["axes"], case["positions"]
    t = torch.arange(T, device=dev)
    if case["prompts"]:
        p = t % -(-T // case["prompts"])
        if A > 1:    # frames of 24 x 32
            p = torch.stack((p // 768, p // 32 % 24, p % 32))[3 - A:]
        else:
            p = p[None]
        p = p + torch.randint(0, P - T, (A, 1), generator=gen, device=dev) if T < P // 2 else p
    else:
        p = torch.randint(0, P, (A, T), generator=gen, device=dev)
    return (p % P).to(torch.int32).contiguous()


def _axis(case, dev):
    """The axis whose position each frequency takes, uint8: runs of frequencies, or in turn."""
    A, n = case["axes"], case["rotary_dim"] // 2
    f = np.arange(n)
    if case["sections"]:
        a = np.searchsorted(np.cumsum([n // 4, (3 * n) // 8]), f, side="right") if A == 3 else (
            f * A // n)
    else:
        a = f % A
    return torch.from_numpy(a.astype(np.uint8)).to(dev) if A > 1 else None


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    H, G, d = case["heads"], case["kv_heads"], case["head_dim"]
    s = {"case": dict(case)}
    if case["kind"] == "prompt":
        lens = _lens(case)
        T = int(lens.sum())
        s["q"], s["k"], s["v"] = _projection(case, T, gen, dev)
        start = np.concatenate([[0], np.cumsum(lens)])
        s["start"] = torch.from_numpy(start.astype(np.int32)).to(dev)
        s["max_len"] = int(lens.max())
        s["out"] = torch.empty((T, H, d), dtype=dtype, device=dev)
        # the plan of a padded batch: which token each (prompt, place) is, and back
        i = np.minimum(np.arange(lens.max())[None, :], lens[:, None] - 1)
        s["token_of"] = torch.from_numpy(start[:-1, None] + i).to(dev)
        s["row_of"] = torch.from_numpy(np.concatenate(
            [b * lens.max() + np.arange(n) for b, n in enumerate(lens)])).to(dev)
        return s
    T = case["tokens"]
    s["q"], s["k"], s["v"] = _projection(case, T, gen, dev)
    s["table"] = _table(case["rotary_dim"], case["positions"], dev)
    s["pos"] = _positions(case, gen, dev)
    s["axis"] = _axis(case, dev)
    s["q_out"] = torch.zeros((T, H, d), dtype=dtype, device=dev)
    if case["kind"] == "rope":
        s["k_out"] = torch.zeros((T, G, d), dtype=dtype, device=dev)
        return s
    pool = T // BLOCK + T // 64 + 9 if case["prompts"] else T + T // 8 + 9
    s["pool"] = pool
    if case["prompts"]:   # whole blocks in scattered order
        blocks = torch.randperm(pool, generator=gen, device=dev)
        t = torch.arange(T, device=dev)
        slots = blocks[t // BLOCK] * BLOCK + t % BLOCK
    else:                 # one slot in a block of its own each
        slots = (torch.randperm(pool, generator=gen, device=dev)[:T] * BLOCK +
                 torch.randint(0, BLOCK, (T,), generator=gen, device=dev))
    if case["padded"]:
        slots[T - case["padded"]:] = -1
    s["slots"] = slots.long()
    kind = case["cache"]
    width = d // 2 if kind == "int4" else d
    kv = {"int4": torch.uint8, "int8": torch.int8, "fp8": torch.float8_e4m3fn}.get(kind, dtype)
    for n in ("k", "v"):
        s[n + "_cache"] = torch.zeros((pool, G, BLOCK, width), dtype=torch.uint8 if kind == "fp8"
                                      else kv, device=dev).view(kv)
        s[n + "_scale"] = s[n + "_zp"] = None
        if kind in ("int4", "int8"):
            row = (pool, G, BLOCK) + ((d // GROUP,) if kind == "int4" else ())
            s[n + "_scale"] = torch.zeros(row, device=dev)
            s[n + "_zp"] = torch.zeros(row, dtype=torch.int8, device=dev)
        if kind == "fp8":   # calibrated a head each: about the largest value at the code 448
            s[n + "_scale"] = (20.0 + torch.rand((G,), generator=gen, device=dev)) / 448.0
        if kind != case["dtype"]:
            s[n + "_read"] = torch.zeros((T, G, d), dtype=dtype, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _cos_sin(s):
    """cos and sin of every token and frequency, fp32 [T, 1, rotary_dim / 2]."""
    n = s["case"]["rotary_dim"] // 2
    f = torch.arange(n, device=s["table"].device)
    p = s["pos"].long()
    p = p[s["axis"].long()].t() if s["axis"] is not None else p.t()    # [T, n] or [T, 1]
    return s["table"][p, f][:, None], s["table"][p, f + n][:, None]


def _rotate(x, cos, sin, case):
    """Rows [T, heads, d] rotated, fp32."""
    x = x.float()
    rd = case["rotary_dim"]
    y, tail = x[..., :rd], x[..., rd:]
    if case["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
    else:
        a, b = y[..., :rd // 2], y[..., rd // 2:]
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((y, tail), -1) if rd < x.shape[-1] else y


def _plain_rope(s):
    cos, sin = _cos_sin(s)
    if s["case"]["inverse"]:
        sin = -sin
    s["q_out"] = _rotate(s["q"], cos, sin, s["case"]).to(s["q"].dtype)
    s["k_out"] = _rotate(s["k"], cos, sin, s["case"]).to(s["k"].dtype)


def _quantise(x, codes, low):
    """Codes low .. low + codes, scale and zero point of each last axis."""
    mn = x.amin(-1).clamp(max=0)
    mx = x.amax(-1).clamp(min=0)
    # a tensor divisor: division by a Python number is a product with its reciprocal
    scale = (mx - mn) / torch.full((1,), float(codes), device=x.device)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    zp = (low - torch.round(mn / scale)).clamp(low, low + codes)
    code = (torch.round(x / scale[..., None]) + zp[..., None]).clamp(low, low + codes)
    return code, scale, zp


def _plain_append(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    s["q_out"] = _rotate(s["q"], cos, sin, c).to(s["q"].dtype)
    at = s["slots"] >= 0
    slot = s["slots"][at]
    blk, off = slot // BLOCK, slot % BLOCK
    for n, x in (("k", _rotate(s["k"], cos, sin, c)[at]), ("v", s["v"][at].float())):
        if c["cache"] == c["dtype"]:
            s[n + "_cache"][blk, :, off] = x.to(s["q"].dtype)
            continue
        if c["cache"] == "fp8":
            scale = s[n + "_scale"][:, None]
            code = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[n + "_cache"].view(torch.uint8)[blk, :, off] = code.view(torch.uint8)
            value = code.float() * scale
        elif c["cache"] == "int8":
            code, scale, zp = _quantise(x, 255, -128)
            value = (code - zp[..., None]) * scale[..., None]
            s[n + "_cache"][blk, :, off] = code.to(torch.int8)
        else:
            code, scale, zp = _quantise(x.reshape(*x.shape[:-1], -1, GROUP), 15, 0)
            value = ((code - zp[..., None]) * scale[..., None]).flatten(-2)
            code = code.to(torch.uint8).flatten(-2)
            s[n + "_cache"][blk, :, off] = code[..., 0::2] | (code[..., 1::2] << 4)
        if c["cache"] != "fp8":
            s[n + "_scale"][blk, :, off] = scale
            s[n + "_zp"][blk, :, off] = zp.to(torch.int8)
        s[n + "_read"][at] = value.to(s["q"].dtype)


def _plain_prompt(s):
    """A padded batch, a block of queries at a time against the keys up to its end."""
    token, H, G = s["token_of"], s["case"]["heads"], s["case"]["kv_heads"]
    B, L = token.shape
    d, R = s["q"].shape[-1], H // G
    k = s["k"].float()[token].transpose(1, 2)                      # [B, G, L, d]
    v = s["v"].float()[token].transpose(1, 2)
    q = s["q"].float()[token].transpose(1, 2).reshape(B, G, R, L, d)
    step = max(1, min(L, SCORES // (B * H * L)))
    out = []
    for i in range(0, L, step):
        n = min(L, i + step)
        e = q[:, :, :, i:n] @ k[:, :, None, :n].transpose(-1, -2) / math.sqrt(d)
        t = torch.arange(n, device=e.device)
        e = e.masked_fill_(t > t[i:, None], -math.inf)
        e = torch.exp_(e.sub_(e.amax(-1, keepdim=True)))
        out.append(e @ v[:, :, None, :n] / e.sum(-1, keepdim=True))
    o = torch.cat(out, 3).permute(0, 3, 1, 2, 4).reshape(B * L, H, d)
    return o[s["row_of"]].to(s["q"].dtype)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(s):
    import paged_kv_cache_154_gb300 as pa
    c = s["case"]
    if c["kind"] == "prompt":
        pa.prompt_attention(s["out"], s["q"], s["k"], s["v"], s["start"], s["max_len"],
                            1.0 / math.sqrt(c["head_dim"]))
    elif c["kind"] == "rope":
        pa.rope(s["q_out"], s["q"], s["k_out"], s["k"], s["table"], s["pos"],
                interleaved=c["interleaved"], freq_axis=s["axis"], inverse=c["inverse"])
    else:
        cache = (s["k_cache"], s["v_cache"], s["slots"])
        scales = (s["k_scale"], s["v_scale"], s["k_zp"], s["v_zp"])
        pa.rope_append_kv(s["q_out"], s["q"], s["k"], s["v"], *cache, s["table"], s["pos"],
                          s["pool"], *scales, interleaved=c["interleaved"], freq_axis=s["axis"])
        if c["cache"] != c["dtype"]:
            pa.gather_kv(s["k_read"], s["v_read"], *cache, s["pool"], *scales)


def _names(case):
    if case["kind"] == "rope":
        return ("q_out", "k_out")
    if case["cache"] == case["dtype"]:
        return ("q_out", "k_cache", "v_cache")
    more = ("k_scale", "v_scale", "k_zp", "v_zp") if case["cache"] != "fp8" else ()
    return ("q_out", "k_read", "v_read") + more


def run(state):
    s = state
    kind = s["case"]["kind"]
    if own:
        _own(s)
    elif kind == "prompt":
        return {"out": _plain_prompt(s)}
    else:
        {"rope": _plain_rope, "append": _plain_append}[kind](s)
    if kind == "prompt":
        return {"out": s["out"]}
    return {n: s[n] for n in _names(s["case"])}


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------

def work(case):
    H, G, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["kind"] == "prompt":
        lens = _lens(case)
        pairs = int((lens * (lens + 1) // 2).sum())
        return {"bytes": 4 * int(lens.sum()) * (H + G) * d + 4 * (len(lens) + 1),
                "flops": 4 * d * H * pairs}
    T, rd = case["tokens"], case["rotary_dim"]
    # rows of the table that are met: a prompt's positions, again for every prompt
    rows = -(-T // case["prompts"]) if case["prompts"] and case["axes"] == 1 else T
    table = 4 * rd * min(rows, case["positions"]) + 4 * case["axes"] * T
    flops = 3 * rd * T * (H + G)
    if case["kind"] == "rope":
        return {"bytes": 4 * T * (H + G) * d + table, "flops": flops}
    n = (T - case["padded"]) * G
    row = {"int4": d // 2 + 5 * (d // GROUP), "int8": d + 5, "fp8": d}.get(case["cache"], 2 * d)
    read = 0 if case["cache"] == case["dtype"] else row + 2 * d
    return {"bytes": 4 * T * H * d + n * 2 * (2 * d + row + read) + 8 * T + table,
            "flops": flops + (n * 2 * 6 * d if read else 0)}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_rotated(s, x):
    c, T = s["case"], x.shape[0]
    n = c["rotary_dim"] // 2
    table = s["table"].double()
    y = x.double().clone()
    for f in range(n):
        a = int(s["axis"][f]) if s["axis"] is not None else 0
        p = s["pos"][a].long()
        cos, sin = table[p, f].reshape(T, 1), table[p, n + f].reshape(T, 1)
        if c.get("inverse"):
            sin = -sin
        i, j = (2 * f, 2 * f + 1) if c["interleaved"] else (f, f + n)
        u, w = x[..., i].double(), x[..., j].double()
        y[..., i] = u * cos - w * sin
        y[..., j] = w * cos + u * sin
    return y


def _exact_codes(x, n, low):
    """The values of codes of n + 1 levels a last axis, their scales and zero points."""
    mn, mx = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    scale = (mx - mn) / n
    scale[scale == 0] = 1
    zp = (low - torch.round(mn / scale)).clamp(low, low + n)
    code = (torch.round(x / scale.unsqueeze(-1)) + zp.unsqueeze(-1)).clamp(low, low + n)
    return (code - zp.unsqueeze(-1)) * scale.unsqueeze(-1), scale


def exact(case, seed):
    if case["kind"] == "prompt":
        lens = _lens(case)
        # 64-bit products at about a TFLOP/s
        if 4 * case["head_dim"] * case["heads"] * float((lens.astype(np.float64) ** 2).sum()) > 4e12:
            return None
        s = prepare(case, seed)
        R = case["heads"] // case["kv_heads"]
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=s["out"].device)
        at = 0
        for n in map(int, lens):
            t = torch.arange(n, device=out.device)
            for h in range(case["heads"]):
                q = s["q"][at:at + n, h].double()
                k = s["k"][at:at + n, h // R].double()
                w = q @ k.t() * (1.0 / math.sqrt(case["head_dim"]))
                w[t[None, :] > t[:, None]] = -math.inf
                w = torch.exp(w - torch.logsumexp(w, 1, keepdim=True))
                out[at:at + n, h] = w @ s["v"][at:at + n, h // R].double()
            at += n
        return {"out": out}
    s = prepare(case, seed)
    got = {"q_out": _exact_rotated(s, s["q"])}
    k = _exact_rotated(s, s["k"])
    if case["kind"] == "rope":
        return {**got, "k_out": k}
    kind, d = case["cache"], case["head_dim"]
    used = (s["slots"] >= 0).nonzero().flatten()
    slot = s["slots"][used]
    for n, x in (("k", k), ("v", s["v"].double())):
        x = x[used]
        if kind == case["dtype"]:
            flat = torch.zeros((s["pool"] * BLOCK, *x.shape[1:]), dtype=torch.float64,
                               device=x.device)
            flat[slot] = x
            got[n + "_cache"] = flat.reshape(s["pool"], BLOCK, *x.shape[1:]).transpose(1, 2)
            continue
        read = torch.zeros((case["tokens"], *x.shape[1:]), dtype=torch.float64, device=x.device)
        if kind == "fp8":
            scale = s[n + "_scale"].double()[:, None]
            y = (x / scale).clamp(-448, 448)
            # 3 fraction bits above 2^-6, multiples of 2^-9 below
            power = torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent - 1
            step = torch.ldexp(torch.ones_like(y), power - 3)
            read[used] = torch.round(y / step) * step * scale
        else:
            parts = x if kind == "int8" else x.reshape(*x.shape[:-1], d // GROUP, GROUP)
            value, scale = _exact_codes(parts, 255 if kind == "int8" else 15,
                                        -128 if kind == "int8" else 0)
            read[used] = value.reshape(x.shape)
            flat = torch.zeros((s["pool"] * BLOCK, *scale.shape[1:]), dtype=torch.float64,
                               device=x.device)
            flat[slot] = scale
            got[n + "_scale"] = flat.reshape(s["pool"], BLOCK, *scale.shape[1:]).transpose(1, 2)
        got[n + "_read"] = read
    if kind in ("int8", "int4"):
        got["k_zp"] = got["v_zp"] = None    # whole numbers
    return got
