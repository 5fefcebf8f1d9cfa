"""Plain forms of rotary positions and of attention over prompts (test infrastructure).

numpy only, from the definitions: a pair (a, b) of a row at a position becomes
(a cos - b sin, b cos + a sin); a query of a prompt sees the keys of its own
prompt up to its own token.
"""
from __future__ import annotations

import numpy as np

from .compressed import quantise_int4


def table(positions: int, rotary_dim: int, base: float = 10000.0) -> np.ndarray:
    """cos and sin of position / base ^ (2 f / rotary_dim), fp32 [positions, rotary_dim]."""
    f = base ** (-np.arange(0, rotary_dim, 2) / rotary_dim)
    angle = np.arange(positions, dtype=np.float64)[:, None] * f
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def angles(cos_sin: np.ndarray, positions: np.ndarray, freq_axis=None):
    """cos and sin [T, rotary_dim / 2] of every token; positions [axes, T]."""
    n = cos_sin.shape[1] // 2
    axis = np.zeros(n, np.int64) if freq_axis is None else np.asarray(freq_axis, np.int64)
    f = np.arange(n)
    at = np.asarray(positions)[axis].T                       # [T, n]
    return cos_sin[at, f], cos_sin[at, n + f]


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool = False,
           dtype=np.float64) -> np.ndarray:
    """Rows [T, heads, d] rotated, every product and sum in `dtype`."""
    y = x.astype(dtype)
    n = cos.shape[1]
    first = np.arange(n) * 2 if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    c, s = cos.astype(dtype)[:, None], sin.astype(dtype)[:, None]
    a, b = y[..., first], y[..., second]
    out = y.copy()
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    return out


def quantise_int8(x: np.ndarray):
    """Rows [..., d] fp32 -> int8 codes, fp32 scale and int8 zero point a row."""
    x = np.asarray(x, np.float32)
    mn = np.minimum(x.min(-1), np.float32(0))
    mx = np.maximum(x.max(-1), np.float32(0))
    scale = ((mx - mn) / np.float32(255)).astype(np.float32)
    scale[scale == 0] = 1
    zp = np.clip(np.float32(-128) - np.rint(mn / scale), -128, 127)
    code = np.clip(np.rint(x / scale[..., None]) + zp[..., None], -128, 127)
    return code.astype(np.int8), scale, zp.astype(np.int8)


def quantise(x: np.ndarray, kind: str):
    return quantise_int4(x) if kind == "int4" else quantise_int8(x)


def prompt_attention(q, k, v, lens, scale: float) -> np.ndarray:
    """float64 [T, H, d] of packed prompts: q [T, H, d], k and v [T, H_kv, d]; rows behind
    the last prompt are 0."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out = np.zeros(q.shape)
    group = q.shape[1] // k.shape[1]
    at = 0
    for n in lens:
        n = int(n)
        for h in range(q.shape[1] if n else 0):
            g = h // group
            s = q[at:at + n, h] @ k[at:at + n, g].T * scale
            s[np.triu_indices(n, 1)] = -np.inf
            w = np.exp(s - s.max(1, keepdims=True))
            # a masked token adds nothing, whatever its row holds
            w /= w.sum(1, keepdims=True)
            out[at:at + n, h] = w @ v[at:at + n, g]
        at += n
    return out
