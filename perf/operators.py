"""The cache-compression operators of the paged KV cache, as cases to be measured.

Four operators, each on the library's paged layout (16-token blocks, a block
table per sequence, [num_blocks][num_kv_heads][16][...] arrays):

* "append":  K/V rows quantised to 4 bits into the cache through a slot mapping
             and read back at the values the cache holds (append_kv, gather_kv);
* "decode":  attention of a decode or verify step over a 4-bit cache (decode);
* "weights": the attention weight each cached token received from a run of
             queries, added to its accumulated weight (accumulate_weights);
* "evict":   the tokens of least accumulated weight leave the cache: the kept
             ones are chosen per KV head, and those behind the new length move
             into the holes before it (evict_select, move_tokens).

Where `own` is false, `run` computes them with elementary torch operations in
32 bits; where it is true, with the library's calls.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16     # tokens per cache block
GROUP = 64     # elements that share a 4-bit scale and zero point
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step's new token of each of 64 sequences (8 KV heads), two padded rows
        {"name": "append_step", "kind": "append", "tokens": 66, "padded": 2, "kv_heads": 8,
         "head_dim": 128, "dtype": "bf16", "runs": False, "lens_seed": 1},
        # a prefill's chunks: 8 prompts of 2048 tokens written, and read back for the
        # chunk's own attention
        {"name": "append_prefill", "kind": "append", "tokens": 16384, "padded": 0, "kv_heads": 8,
         "head_dim": 128, "dtype": "bf16", "runs": True, "lens_seed": 2},
        # four short sequences, the smallest step: latency
        {"name": "decode_tiny", "kind": "decode", "seqs": 4, "len_lo": 17, "len_hi": 100,
         "heads": 8, "kv_heads": 2, "head_dim": 64, "run_lo": 1, "run_hi": 1, "dtype": "f16",
         "lens_seed": 3},
        # the Llama-3-8B-shaped step: 64 sequences of 512 to 4096 tokens
        {"name": "decode_llama3_8b", "kind": "decode", "seqs": 64, "len_lo": 512, "len_hi": 4096,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "run_lo": 1, "run_hi": 1, "dtype": "bf16",
         "lens_seed": 4},
        # a speculative verify step, Llama-2-70B-shaped: 8 query heads per KV head, 2-5 tokens
        {"name": "decode_verify", "kind": "decode", "seqs": 16, "len_lo": 1000, "len_hi": 8192,
         "heads": 64, "kv_heads": 8, "head_dim": 128, "run_lo": 2, "run_hi": 5, "dtype": "bf16",
         "lens_seed": 5},
        # few very long sequences: the work has to be split along the context
        {"name": "decode_long", "kind": "decode", "seqs": 4, "len_lo": 32768, "len_hi": 131072,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "run_lo": 1, "run_hi": 1, "dtype": "bf16",
         "lens_seed": 6},
        # accumulated weights at every decode step, beside the Llama-3-8B-shaped attention
        {"name": "weights_step", "kind": "weights", "cache": "bf16", "seqs": 64, "len_lo": 512,
         "len_hi": 4096, "heads": 32, "kv_heads": 8, "head_dim": 128, "run_lo": 1, "run_hi": 1,
         "dtype": "bf16", "carry": True, "lens_seed": 7},
        # a prompt scored once, by its last 32 queries, before it is compressed
        {"name": "weights_window", "kind": "weights", "cache": "f16", "seqs": 8, "len_lo": 1000,
         "len_hi": 4001, "heads": 16, "kv_heads": 4, "head_dim": 64, "run_lo": 32, "run_hi": 32,
         "dtype": "f16", "carry": False, "lens_seed": 8},
        # one long 4-bit sequence
        {"name": "weights_long_int4", "kind": "weights", "cache": "int4", "seqs": 1,
         "len_lo": 100001, "len_hi": 100001, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "run_lo": 1, "run_hi": 1, "dtype": "bf16", "carry": True, "lens_seed": 9},
        # a running batch at its budget gives a block of every sequence back
        {"name": "evict_step", "kind": "evict", "seqs": 64, "len_lo": 1041, "len_hi": 1056,
         "budget": 1040, "kv_heads": 8, "head_dim": 128, "sinks": 4, "recent": 128,
         "dtype": "bf16", "again": True, "lens_seed": 10},
        # prompts compressed once to a quarter and less
        {"name": "evict_prompt", "kind": "evict", "seqs": 16, "len_lo": 2000, "len_hi": 8192,
         "budget": 1024, "kv_heads": 8, "head_dim": 128, "sinks": 4, "recent": 64,
         "dtype": "bf16", "again": False, "lens_seed": 11},
        # one long context compressed to a quarter
        {"name": "evict_long", "kind": "evict", "seqs": 1, "len_lo": 131072, "len_hi": 131072,
         "budget": 32768, "kv_heads": 8, "head_dim": 128, "sinks": 16, "recent": 1024,
         "dtype": "f16", "again": False, "lens_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "weights", "weights", "evict", "evict"])
    c = {"kind": kind, "head_dim": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f16"]),
         "lens_seed": rng.randrange(1 << 20)}
    if kind == "append":
        c["kv_heads"] = rng.choice([1, 2, 3, 5, 8])
        c["tokens"] = _log_int(rng, 1, 16384)
        c["padded"] = rng.choice([0, 0, 1, 5]) if c["tokens"] > 8 else 0
        c["runs"] = rng.random() < 0.5
        return c
    c["kv_heads"] = rng.choice([1, 2, 3, 4, 8])
    c["seqs"] = _log_int(rng, 1, 64)
    # (token, KV head) pairs, and query rows on them, up to the largest listed step's work
    pairs, run_hi = 1100000, 1
    if kind != "evict":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        runs = [(1, 1), (1, 1), (1, 3), (2, 5)] if kind == "decode" else [(1, 1), (1, 1), (1, 4),
                                                                          (16, 16)]
        run_lo, run_hi = rng.choice(runs)
        c.update(heads=c["kv_heads"] * group, run_lo=run_lo, run_hi=run_hi)
        pairs = min(pairs, 12000000 // (group * run_hi))
    if kind == "weights":
        c["cache"] = rng.choice(["int4", "int8", "fp8", c["dtype"], c["dtype"]])
        c["carry"] = rng.random() < 0.5
    c["len_hi"] = _log_int(rng, 20, max(20, min(131072, pairs // (c["seqs"] * c["kv_heads"]))))
    c["len_lo"] = max(run_hi, int(c["len_hi"] * rng.choice([0.02, 0.3, 0.9])))
    if kind == "evict":
        c["budget"] = _log_int(rng, 1, c["len_hi"])
        c["sinks"] = rng.choice([0, 1, 4, 16])
        c["recent"] = rng.choice([0, 1, 17, 64])
        c["again"] = rng.random() < 0.5
    return c


def _lens(case):
    """Context lengths and query runs; the case alone decides them."""
    r = np.random.RandomState(case["lens_seed"])
    lens = r.randint(case["len_lo"], case["len_hi"] + 1, case["seqs"])
    runs = r.randint(case.get("run_lo", 1), case.get("run_hi", 1) + 1, case["seqs"])
    return lens.astype(np.int64), np.minimum(runs, lens).astype(np.int64)


# ---------------------------------------------------------------------------
# 4-bit rows: scale = (max - min) / 15 over a group of 64 widened to hold 0,
# zero point = -rint(min / scale), code = rint(x / scale) + zero point, in
# IEEE fp32; byte j of a row holds elements 2j (low half) and 2j + 1
# ---------------------------------------------------------------------------

def _quantise4(x):
    x = x.float().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    mn = x.amin(-1).clamp(max=0)
    mx = x.amax(-1).clamp(min=0)
    # a tensor divisor: division by a Python number is a product with its reciprocal
    scale = (mx - mn) / torch.full((1,), 15.0, device=x.device)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    zp = (-torch.round(mn / scale)).clamp(0, 15)
    code = (torch.round(x / scale[..., None]) + zp[..., None]).clamp(0, 15)
    code = code.to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, zp.to(torch.int8)


def _values4(packed, scale, zp):
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).float()
    g = scale.shape[-1]
    code = code.reshape(*code.shape[:-1], g, code.shape[-1] // g)
    return ((code - zp.float()[..., None]) * scale[..., None]).flatten(-2)


def _quantise8(x):
    x = x.float()
    mn = x.amin(-1).clamp(max=0)
    mx = x.amax(-1).clamp(min=0)
    scale = (mx - mn) / torch.full((1,), 255.0, device=x.device)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    zp = (-128 - torch.round(mn / scale)).clamp(-128, 127)
    code = (torch.round(x / scale[..., None]) + zp[..., None]).clamp(-128, 127)
    return code.to(torch.int8), scale, zp.to(torch.int8)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _tables(case, lens, gen, dev):
    """Blocks of every sequence, spread over a pool a little larger than needed."""
    need = (lens + BLOCK - 1) // BLOCK
    pool = int(need.sum()) + 8
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32).cpu().numpy()
    tables = np.full((len(lens), int(need.max())), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += int(n)
    return pool, torch.from_numpy(tables).to(dev)


def _rows(shape, gen, dev, dtype):
    """K or V rows: normal, with a few channels of a larger range, as caches have."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    x[..., ::29] *= 3.0
    return x.to(dtype)


def _cache(kind, pool, heads, dim, gen, dev, dtype):
    x = _rows((pool, heads, BLOCK, dim), gen, dev, dtype)
    if kind == "int4":
        return _quantise4(x)
    if kind == "int8":
        return _quantise8(x)
    if kind == "fp8":
        scale = x.float().abs().amax((0, 2, 3)) / 448.0
        y = (x.float() / scale[None, :, None, None]).clamp(-448, 448)
        return y.to(torch.float8_e4m3fn), scale, None
    return x, None, None


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    H, d = case["kv_heads"], case["head_dim"]
    s = {"case": dict(case)}
    if case["kind"] == "append":
        T = case["tokens"]
        pool = T // BLOCK + T // 64 + 9 if case["runs"] else 2 * T + 9
        s["pool"] = pool
        if case["runs"]:     # whole blocks in scattered order
            blocks = torch.randperm(pool, generator=gen, device=dev)
            t = torch.arange(T, device=dev)
            slots = blocks[t // BLOCK] * BLOCK + t % BLOCK
        else:                # one slot in a block of its own each
            slots = (torch.randperm(pool, generator=gen, device=dev)[:T] * BLOCK +
                     torch.randint(0, BLOCK, (T,), generator=gen, device=dev))
        if case["padded"]:
            slots[T - case["padded"]:] = -1
        s["slots"] = slots.long()
        s["key"] = _rows((T, H, d), gen, dev, dtype)
        s["value"] = _rows((T, H, d), gen, dev, dtype)
        g = d // GROUP
        for n in ("k", "v"):
            s[n] = torch.zeros((pool, H, BLOCK, d // 2), dtype=torch.uint8, device=dev)
            s[n + "_scale"] = torch.zeros((pool, H, BLOCK, g), device=dev)
            s[n + "_zp"] = torch.zeros((pool, H, BLOCK, g), dtype=torch.int8, device=dev)
            s[n + "_out"] = torch.zeros((T, H, d), dtype=dtype, device=dev)
        return s
    lens, runs = _lens(case)
    S, Lm = len(lens), int(lens.max())
    s["pool"], s["tables"] = _tables(case, lens, gen, dev)
    s["max_len"] = Lm
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
    kind = {"decode": "int4", "evict": case["dtype"]}.get(case["kind"], case.get("cache"))
    s["k"], s["k_scale"], s["k_zp"] = _cache(kind, s["pool"], H, d, gen, dev, dtype)
    if case["kind"] != "weights":
        s["v"], s["v_scale"], s["v_zp"] = _cache(kind, s["pool"], H, d, gen, dev, dtype)
    if case["kind"] == "evict":
        kept = np.minimum(lens, case["budget"]).astype(np.int32)
        s["new_lens"] = torch.from_numpy(kept).to(dev)
        w = torch.exp(2 * torch.randn((S, H, Lm), generator=gen, device=dev))
        # tokens that never got a weight worth a float: exact ties
        w[torch.rand((S, H, Lm), generator=gen, device=dev) < 0.1] = 0
        s["scores"] = w
        pos = torch.full((S, H, Lm), -1, dtype=torch.int32, device=dev)
        total = lens.astype(np.int64)
        if case["again"]:    # evicted before: the first tokens stand in no order
            n = min(case["budget"], int(lens.min())) // 2
            total = total + n
            if n:
                pos[..., :n] = torch.rand((S, H, 2 * n), generator=gen, device=dev).argsort(
                    -1)[..., :n].to(torch.int32)
        s["positions"] = pos
        s["total_lens"] = torch.from_numpy(total.astype(np.int32)).to(dev)
        s["scores_out"] = torch.zeros_like(w)
        s["positions_out"] = torch.zeros_like(pos)
        s["moves"] = torch.zeros((S, H, max(1, Lm // 2), 2), dtype=torch.int32, device=dev)
        s["counts"] = torch.zeros((S, H), dtype=torch.int32, device=dev)
        return s
    nq, Hq = int(runs.sum()), case["heads"]
    start = np.concatenate([[0], np.cumsum(runs)])
    s["start"] = torch.from_numpy(start.astype(np.int32)).to(dev) if runs.max() > 1 else None
    s["max_run"] = int(runs.max())
    s["scale"] = 1.0 / math.sqrt(d)
    s["q"] = torch.randn((nq, Hq, d), generator=gen, device=dev).to(dtype)
    s["out"] = torch.empty((nq, Hq, d), dtype=dtype, device=dev)
    # the plan of a padded batch: which token each (sequence, query) is, and back
    s["runs"] = torch.from_numpy(runs).to(dev)
    i = np.minimum(np.arange(runs.max())[None, :], runs[:, None] - 1)
    s["token_of"] = torch.from_numpy(start[:-1, None] + i).to(dev)
    s["row_of"] = torch.from_numpy(np.concatenate(
        [b * runs.max() + np.arange(r) for b, r in enumerate(runs)])).to(dev)
    if case["kind"] == "weights":
        s["scores"] = (torch.rand((S, H, Lm), generator=gen, device=dev) * 4
                       if case["carry"] else None)
        s["scores_out"] = torch.zeros((S, H, Lm), device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _dense(s, n):
    """A cache's values as every sequence's tokens, [S, H, tokens, d] fp32."""
    idx = s["tables"].long().clamp(min=0)

    def tokens(x):
        x = x[idx].transpose(1, 2)                      # [S, H, blocks, 16, ...]
        return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])

    x = tokens(s[n])
    if x.dtype == torch.uint8:
        return _values4(x, tokens(s[n + "_scale"]), tokens(s[n + "_zp"]))
    if x.dtype == torch.int8:
        return (x.float() - tokens(s[n + "_zp"]).float()[..., None]) * tokens(
            s[n + "_scale"])[..., None]
    if s[n + "_scale"] is not None:
        return x.float() * s[n + "_scale"][None, :, None, None]
    return x.float()


def _softmax(s):
    """exp(logit - max) of every (sequence, KV head, query row, token), 0 where masked, and
    its sums; a row is query i of the run and head h of the group, i * group + h."""
    S, H = s["tables"].shape[0], s["case"]["kv_heads"]
    R, G = s["token_of"].shape[1], s["case"]["heads"] // H
    q = s["q"].float()[s["token_of"]].reshape(S, R, H, G, -1).transpose(1, 2)
    k = _dense(s, "k")
    logits = q.reshape(S, H, R * G, -1) @ k.transpose(2, 3) * s["scale"]
    i = torch.arange(R, device=q.device)
    lens, runs = s["lens"].long(), s["runs"]
    last = lens[:, None] - runs[:, None] + i            # last token that query i sees
    last = torch.where(i < runs[:, None], last, torch.full_like(last, -1))
    t = torch.arange(k.shape[2], device=q.device)
    seen = (t <= last[..., None]).repeat_interleave(G, 1)[:, None]
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return e, e.sum(-1, keepdim=True)


def _plain_append(s):
    at = s["slots"] >= 0
    slot = s["slots"][at]
    blk, off = slot // BLOCK, slot % BLOCK
    for n, x in (("k", s["key"]), ("v", s["value"])):
        for a, y in zip((s[n], s[n + "_scale"], s[n + "_zp"]), _quantise4(x[at])):
            a[blk, :, off] = y
        s[n + "_out"][at] = _values4(s[n][blk, :, off], s[n + "_scale"][blk, :, off],
                                     s[n + "_zp"][blk, :, off]).to(x.dtype)


def _plain_decode(s):
    e, total = _softmax(s)
    o = (e @ _dense(s, "v")) / total                    # [S, H, R * G, d]
    S, H, R = o.shape[0], o.shape[1], s["token_of"].shape[1]
    o = o.reshape(S, H, R, -1, o.shape[-1]).transpose(1, 2).reshape(S * R, -1, o.shape[-1])
    return o[s["row_of"]].to(s["q"].dtype)


def _plain_weights(s):
    e, total = _softmax(s)
    w = torch.where(total > 0, e / total, torch.zeros_like(e)).sum(2)[..., :s["max_len"]]
    if s["scores"] is not None:
        w = w + s["scores"]
    inside = torch.arange(s["max_len"], device=w.device) < s["lens"].long()[:, None, None]
    s["scores_out"] = torch.where(inside, w, s["scores_out"])


def _plain_evict(s):
    c = s["case"]
    w, L, n = s["scores"], s["lens"].long()[:, None, None], s["new_lens"].long()[:, None, None]
    total = s["total_lens"].long()[:, None, None]
    slot = torch.arange(w.shape[2], device=w.device).expand(w.shape)
    pos = s["positions"].long()
    pos = torch.where(pos >= 0, pos, total - L + slot)
    safe = (pos < c["sinks"]) | (pos >= total - c["recent"])
    key = torch.where(safe, torch.full_like(w, math.inf), w)
    key = torch.where(slot < L, key, torch.full_like(w, -math.inf))
    rank = key.argsort(dim=-1, descending=True, stable=True).argsort(dim=-1)
    keep = rank < n
    hole, mover = ~keep & (slot < n), keep & (slot >= n)
    s["counts"] = hole.sum(-1).to(torch.int32)
    # the i-th hole takes the i-th token behind the new length
    b, g, dst = hole.nonzero(as_tuple=True)
    src = mover.nonzero(as_tuple=True)[2]
    i = (hole.cumsum(-1) - 1)[b, g, dst]
    s["moves"][b, g, i, 0] = src.to(torch.int32)
    s["moves"][b, g, i, 1] = dst.to(torch.int32)
    for name, x, gone in (("scores_out", w, 0), ("positions_out", pos.to(torch.int32), -1)):
        y = x.clone()
        y[b, g, dst] = x[b, g, src]
        y = torch.where(slot < n, y, torch.full_like(y, gone))
        s[name] = torch.where(slot < L, y, s[name])
    t = s["tables"].long()
    for name in ("k", "v"):
        x = s[name]
        x[t[b, dst // BLOCK], g, dst % BLOCK] = x[t[b, src // BLOCK], g, src % BLOCK]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

_scratch = {}


def _workspace(kind, nbytes):
    """The scratch memory that a program keeps for all its calls of one kind."""
    w = _scratch.get(kind)
    if nbytes and (w is None or w.numel() < nbytes):
        w = _scratch[kind] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    return w if nbytes else None


def _own(s):
    import paged_kv_cache_154_gb300 as pa
    c = s["case"]
    if c["kind"] == "append":
        cache = (s["k"], s["v"], s["slots"], s["pool"], s["k_scale"], s["v_scale"], s["k_zp"],
                 s["v_zp"])
        pa.append_kv(s["key"], s["value"], *cache)
        pa.gather_kv(s["k_out"], s["v_out"], *cache)
        return
    if c["kind"] == "evict":
        pa.evict_select(s["moves"], s["counts"], s["scores_out"], s["positions_out"],
                        s["scores"], s["positions"], s["lens"], s["new_lens"], s["total_lens"],
                        s["max_len"], c["sinks"], c["recent"])
        pa.move_tokens(s["k"], s["v"], s["tables"], s["lens"], s["moves"], s["counts"],
                       s["max_len"], s["pool"])
        return
    size = (s["tables"].shape[0], s["q"].shape[0], c["heads"], c["kv_heads"], c["head_dim"],
            s["max_run"], s["max_len"])
    if c["kind"] == "decode":
        pa.decode(s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens"], s["max_len"],
                  s["scale"], s["start"], s["max_run"], s["pool"], s["k_scale"], s["v_scale"],
                  s["k_zp"], s["v_zp"], 0, _workspace("decode", pa.decode_workspace_size(*size)))
        return
    pa.accumulate_weights(s["scores_out"], s["scores"], s["q"], s["k"], s["tables"], s["lens"],
                          s["max_len"], s["scale"], s["start"], s["max_run"], s["pool"],
                          s["k_scale"], s["k_zp"],
                          _workspace("weights", pa.accumulate_weights_workspace_size(*size)))


def run(state):
    s = state
    kind = s["case"]["kind"]
    if own:
        _own(s)
    elif kind == "decode":
        return {"out": _plain_decode(s)}
    else:
        {"append": _plain_append, "weights": _plain_weights, "evict": _plain_evict}[kind](s)
    names = {"append": ("k_out", "v_out", "k_scale", "v_scale", "k_zp", "v_zp"),
             "decode": ("out",), "weights": ("scores_out",),
             "evict": ("moves", "counts", "scores_out", "positions_out", "k", "v")}[kind]
    return {n: s[n] for n in names}


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------

def work(case):
    H, d = case["kv_heads"], case["head_dim"]
    row4 = d // 2 + 5 * (d // GROUP)
    if case["kind"] == "append":
        T = case["tokens"]
        n = (T - case["padded"]) * H
        # rows in, the cache's form out and in, rows out; K and V
        return {"bytes": n * 2 * (2 * d + 2 * row4 + 2 * d) + 8 * T, "flops": n * 2 * 6 * d}
    lens, runs = _lens(case)
    tables = 4 * int(((lens + BLOCK - 1) // BLOCK).sum())
    tokens = int(lens.sum()) * H
    if case["kind"] == "evict":
        kept = np.minimum(lens, case["budget"])
        moved = int((kept * (lens - kept) / lens).sum()) * H      # as many as a random choice moves
        return {"bytes": 16 * tokens + 8 * moved + moved * 2 * 2 * 2 * d + tables,
                "flops": 4 * tokens}
    nq, Hq = int(runs.sum()), case["heads"]
    scored = int((lens * runs).sum()) * Hq
    if case["kind"] == "decode":
        return {"bytes": tokens * 2 * row4 + 2 * nq * Hq * d * 2 + tables, "flops": 4 * scored * d}
    row = {"int4": row4, "int8": d + 5, "fp8": d}.get(case["cache"], 2 * d)
    return {"bytes": tokens * (row + (8 if case["carry"] else 4)) + nq * Hq * d * 2 + tables,
            "flops": scored * (2 * d + 4)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _value_rows(s, n, blk, g):
    """float64 values of blocks `blk` (in order) of one KV head, [16 * blocks, d]."""
    x = s[n][blk, g]
    if x.dtype == torch.uint8:
        lo, hi = (x % 16).double(), (x // 16).double()
        y = torch.empty((*x.shape[:2], 2 * x.shape[2]), dtype=torch.float64, device=x.device)
        y[..., 0::2], y[..., 1::2] = lo, hi
        sc, zp = s[n + "_scale"][blk, g].double(), s[n + "_zp"][blk, g].double()
        for j in range(sc.shape[-1]):
            part = y[..., j * GROUP:(j + 1) * GROUP]
            part -= zp[..., j, None]
            part *= sc[..., j, None]
    elif x.dtype == torch.int8:
        y = (x.double() - s[n + "_zp"][blk, g].double()[..., None]) * \
            s[n + "_scale"][blk, g].double()[..., None]
    else:
        y = x.double()
        if s[n + "_scale"] is not None:
            y = y * s[n + "_scale"][g].double()
    return y.reshape(-1, y.shape[-1])


def _exact_attention(case, s):
    lens, runs = _lens(case)
    H, G = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    w = s["scores_out"].double() if case["kind"] == "weights" else None
    first = 0
    for b, (L, r) in enumerate(zip(lens.tolist(), runs.tolist())):
        blk = s["tables"][b, :(L + BLOCK - 1) // BLOCK].long()
        for g in range(H):
            k = _value_rows(s, "k", blk, g)[:L]
            q = s["q"][first:first + r, g * G:(g + 1) * G].double()      # [r, G, d]
            z = torch.einsum("igd,td->igt", q, k) / math.sqrt(case["head_dim"])
            for i in range(r):
                z[i, :, L - r + i + 1:] = -math.inf
            p = torch.softmax(z, -1)
            if w is None:
                out[first:first + r, g * G:(g + 1) * G] = torch.einsum(
                    "igt,td->igd", p, _value_rows(s, "v", blk, g)[:L])
            else:
                w[b, g, :L] = p.sum((0, 1))
                if s["scores"] is not None:
                    w[b, g, :L] += s["scores"][b, g, :L].double()
        first += r
    return {"out": out} if w is None else {"scores_out": w}


def _exact_append(case, s):
    """The quantiser's own definition: each of its operations rounds to fp32, so the stored
    scale, zero point and code are fixed numbers; the values are code - zero point times scale."""
    got = {}
    slots = s["slots"].cpu().numpy()
    f4 = np.float32
    for n, x in (("k", s["key"]), ("v", s["value"])):
        x = x.float().cpu().numpy()
        scales, zps = s[n + "_scale"].cpu().numpy(), s[n + "_zp"].cpu().numpy().astype(np.int64)
        out = np.zeros(x.shape)
        use = np.flatnonzero(slots >= 0)
        for j in range(case["head_dim"] // GROUP):
            part = x[use, :, j * GROUP:(j + 1) * GROUP]
            lo, hi = np.minimum(part.min(-1), f4(0)), np.maximum(part.max(-1), f4(0))
            sc = ((hi - lo) / f4(15)).astype(f4)
            sc[sc == 0] = f4(1)
            zp = np.clip(-np.rint(lo / sc), 0, 15)
            code = np.clip(np.rint(part / sc[..., None]) + zp[..., None], 0, 15)
            out[use, :, j * GROUP:(j + 1) * GROUP] = (
                (code - zp[..., None]).astype(np.float64) * sc[..., None].astype(np.float64))
            scales[slots[use] // BLOCK, :, slots[use] % BLOCK, j] = sc
            zps[slots[use] // BLOCK, :, slots[use] % BLOCK, j] = zp.astype(np.int64)
        got[n + "_out"], got[n + "_scale"], got[n + "_zp"] = out, scales.astype(np.float64), zps
    return got


def _exact_evict(case, s):
    lens, _ = _lens(case)
    w, pos_in = s["scores"].cpu().numpy(), s["positions"].cpu().numpy()
    total, kept = s["total_lens"].cpu().numpy(), s["new_lens"].cpu().numpy()
    moves, counts = s["moves"].cpu().numpy(), s["counts"].cpu().numpy()
    w_out, pos_out = s["scores_out"].double().cpu().numpy(), s["positions_out"].cpu().numpy()
    tables = s["tables"].cpu().numpy()
    caches = [s["k"].double(), s["v"].double()]
    for b, L in enumerate(lens.tolist()):
        n = int(kept[b])
        for g in range(case["kv_heads"]):
            pos = pos_in[b, g, :L].astype(np.int64)
            pos = np.where(pos < 0, total[b] - L + np.arange(L), pos)
            safe = (pos < case["sinks"]) | (pos >= total[b] - case["recent"])
            # the protected ones first, in slot order; then by weight, equal ones in slot order
            weight = np.where(safe, 0.0, w[b, g, :L].astype(np.float64))
            order = np.lexsort((np.arange(L), -weight, ~safe))
            stay = np.zeros(L, bool)
            stay[order[:n]] = True
            dst = np.flatnonzero(~stay[:n])
            src = np.flatnonzero(stay[n:]) + n
            counts[b, g] = len(dst)
            moves[b, g, :len(dst), 0], moves[b, g, :len(dst), 1] = src, dst
            w_out[b, g, :L] = 0
            w_out[b, g, :n] = w[b, g, :n]
            w_out[b, g, dst] = w[b, g, src]
            pos_out[b, g, :L] = -1
            pos_out[b, g, :n] = pos[:n]
            pos_out[b, g, dst] = pos[src]
            fb, tb = tables[b, src // BLOCK], tables[b, dst // BLOCK]
            for x in caches:
                x[tb, g, dst % BLOCK] = x[fb, g, src % BLOCK]
    return {"moves": moves, "counts": counts, "scores_out": w_out, "positions_out": pos_out,
            "k": caches[0], "v": caches[1]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "append":
        return _exact_append(case, s)
    if case["kind"] == "evict":
        return _exact_evict(case, s)
    return _exact_attention(case, s)
