"""Plain 64-bit forms of the cache-compression operators (test infrastructure).

numpy only, one (sequence, KV head) at a time, from the definitions:

  * the INT4 quantiser of "cs336 lecture 10" (Quantization, x_q = round(x/scale)
    + zero_point) with 16 codes and a scale per group of 64 elements;
  * softmax(q k^T scale) v and its weights over the values a cache holds;
  * eviction: which tokens a budget keeps, and the moves that close the holes.
"""
from __future__ import annotations

import numpy as np

GROUP = 64


def quantise_int4(x: np.ndarray):
    """x [..., d] fp32 -> packed uint8 [..., d/2], scale fp32 and zero point
    int8 [..., d/64]; every operation rounds to fp32, as the definition does."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    mn = np.minimum(g.min(-1), np.float32(0))
    mx = np.maximum(g.max(-1), np.float32(0))
    scale = ((mx - mn) / np.float32(15)).astype(np.float32)
    scale[scale == 0] = 1
    zp = np.clip(-np.rint(mn / scale), 0, 15)
    code = np.clip(np.rint(g / scale[..., None]) + zp[..., None], 0, 15)
    code = code.astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, zp.astype(np.int8)


def values_int4(packed: np.ndarray, scale: np.ndarray, zp: np.ndarray) -> np.ndarray:
    """float64 values (code - zero point) * scale."""
    code = np.empty((*packed.shape[:-1], packed.shape[-1] * 2))
    code[..., 0::2], code[..., 1::2] = packed & 15, packed >> 4
    rep = GROUP
    with np.errstate(invalid="ignore"):      # slots of no token may hold infinite scales
        return (code - np.repeat(zp.astype(np.float64), rep, -1)) * np.repeat(
            scale.astype(np.float64), rep, -1)


def cache_values(cache) -> tuple:
    """(K, V) float64 [blocks, H_kv, 16, d] of an engine.PagedKVCache's tensors."""
    import torch
    out = []
    for n in ("k", "v"):
        x = getattr(cache, n).cpu()
        sc = getattr(cache, n + "_scale")
        zp = getattr(cache, n + "_zp")
        sc = None if sc is None else sc.cpu().numpy().astype(np.float64)
        zp = None if zp is None else zp.cpu().numpy()
        if x.dtype == torch.uint8:
            out.append(values_int4(x.numpy(), sc, zp))
        elif x.dtype == torch.int8:
            out.append((x.numpy().astype(np.float64) - zp[..., None]) * sc[..., None])
        elif sc is not None:
            out.append(x.float().double().numpy() * sc[None, :, None, None])
        else:
            out.append(x.double().numpy())
    return tuple(out)


def tokens_of(values: np.ndarray, table, L: int, g: int) -> np.ndarray:
    """[L, d] rows of one sequence and KV head."""
    nb = (L + 15) // 16
    return values[np.asarray(table)[:nb], g].reshape(-1, values.shape[-1])[:L]


def probabilities(q: np.ndarray, k: np.ndarray, scale: float) -> np.ndarray:
    """softmax weights [r, G, L] of a run of r queries q [r, G, d] whose last is
    the last token: query i sees keys 0 .. L - r + i. A query that sees none has
    weights 0."""
    r, L = q.shape[0], k.shape[0]
    z = np.einsum("igd,td->igt", q, k) * scale
    seen = np.arange(L)[None, :] <= (L - r + np.arange(r))[:, None]
    z = np.where(seen[:, None], z, -np.inf)
    m = z.max(-1, keepdims=True) if L else np.zeros((r, q.shape[1], 1))
    e = np.exp(z - np.where(np.isfinite(m), m, 0))
    total = e.sum(-1, keepdims=True)
    return np.where(total > 0, e / np.where(total > 0, total, 1), 0)


def attend(q, k_values, v_values, tables, lens, qsl, scale) -> np.ndarray:
    """[num_q, H, d] float64 attention over cache values (as cache_values gives them)."""
    H_kv = k_values.shape[1]
    G = q.shape[1] // H_kv
    out = np.full(q.shape, np.nan)
    for s, L in enumerate(lens):
        a, b = qsl[s], qsl[s + 1]
        for g in range(H_kv):
            p = probabilities(q[a:b, g * G:(g + 1) * G], tokens_of(k_values, tables[s], L, g),
                              scale)
            out[a:b, g * G:(g + 1) * G] = np.einsum("igt,td->igd", p,
                                                    tokens_of(v_values, tables[s], L, g))
    return out


def weights(q, k_values, tables, lens, qsl, scale, width: int) -> np.ndarray:
    """[S, H_kv, width] float64: the weight each token gets from its sequence's
    queries, summed over the query heads of the group (0 past the context)."""
    H_kv = k_values.shape[1]
    G = q.shape[1] // H_kv
    w = np.zeros((len(lens), H_kv, width))
    for s, L in enumerate(lens):
        a, b = qsl[s], qsl[s + 1]
        for g in range(H_kv):
            if L and b > a:
                w[s, g, :L] = probabilities(q[a:b, g * G:(g + 1) * G],
                                            tokens_of(k_values, tables[s], L, g),
                                            scale).sum((0, 1))
    return w


def select(score: np.ndarray, positions: np.ndarray, L: int, new_len: int, total: int,
           sinks: int, recent: int):
    """One (sequence, KV head): (moves [n, 2] of (source, destination) slots,
    scores [L], positions [L]) after the eviction that keeps new_len tokens.

    A token's position is its entry of `positions`, or total - L + slot where
    that is negative. Kept first: the tokens at positions < sinks or >= total -
    recent, in slot order; then by score, the highest first, NaN last, equal
    ones in slot order. The i-th evicted slot before new_len takes the i-th
    kept token behind it."""
    slot = np.arange(L)
    pos = np.where(positions[:L] >= 0, positions[:L], total - L + slot).astype(np.int64)
    n = L if new_len < 0 else min(new_len, L)
    safe = (pos < sinks) | (pos >= total - recent)
    w = score[:L].astype(np.float64)
    kind = np.where(safe, 0, np.where(np.isnan(w), 2, 1))
    order = np.lexsort((slot, np.where(kind == 1, -w, 0.0), kind))
    keep = np.zeros(L, bool)
    keep[order[:n]] = True
    dst = np.flatnonzero(~keep[:n])
    src = np.flatnonzero(keep[n:]) + n
    s_out, p_out = np.zeros(L, score.dtype), np.full(L, -1, np.int64)
    s_out[:n], p_out[:n] = score[:n], pos[:n]
    s_out[dst], p_out[dst] = score[src], pos[src]
    return np.stack([src, dst], -1), s_out, p_out
