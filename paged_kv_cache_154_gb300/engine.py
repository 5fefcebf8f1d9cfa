"""A paged KV cache for one attention layer, driven through the C ABI.

Holds the device cache tensors (torch allocations: the library itself
allocates nothing) and a host block pool, and runs the decode step in the
order the method requires: reserve slots in the pool (copy-on-write pairs
come back), copy the shared blocks, append the new K/V through the slot
mapping, then attend ("cs336 lecture 10", decode workflow: append the new
K, V, then score q against the cache).

Operations are duck-typed objects: one with `parent`/`child` is a fork, one
with `k`/`v` appends those rows to `seq`, anything else with `seq` creates a
sequence. Names are caller-chosen; `names` maps them to pool ids.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence

import numpy as np
import torch

from . import (BLOCK_SIZE, INT4_GROUP, Pool, accumulate_weights,
               accumulate_weights_workspace_size, append_kv, copy_blocks, decode,
               decode_shared_prefix, decode_shared_prefix_workspace_size, decode_workspace_size,
               evict_select, move_tokens, prompt_attention, prompt_attention_workspace_size,
               rope_append_kv, zeroed_workspace)

KV_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8,
            "fp8": torch.float8_e4m3fn, "int4": torch.uint8}


def rope_table(positions: int, rotary_dim: int, base: float = 10000.0, inv_freq=None,
               factor: float = 1.0, device="cuda") -> torch.Tensor:
    """cos_sin for rope() and rope_append_kv(), fp32 [positions, rotary_dim]: angles of
    position * inv_freq in 64 bits (far positions lose nothing), their cosines and sines
    times `factor` (of scaled rotations) rounded once. inv_freq: rotary_dim / 2 frequencies,
    base ** (-2 f / rotary_dim) without it."""
    if inv_freq is None:
        inv_freq = base ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    f = torch.as_tensor(np.asarray(inv_freq, np.float64), device=device)
    if f.shape != (rotary_dim // 2,) or rotary_dim % 2:
        raise ValueError(f"inv_freq is {tuple(f.shape)}, rotary_dim {rotary_dim}")
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return (torch.cat((angle.cos(), angle.sin()), 1) * factor).float()


@dataclass
class Rotary:
    """How a step's queries and keys are rotated on their way into the cache."""
    cos_sin: torch.Tensor             # fp32 [positions, rotary_dim], as rope_table() makes it
    interleaved: bool = False
    freq_axis: Optional[torch.Tensor] = None   # uint8 [rotary_dim / 2], with several position axes


@dataclass
class StepInputs:
    """Device tensors of one decode step (built once, reusable)."""
    key: torch.Tensor                 # [T, H_kv, d] rows appended this step
    value: torch.Tensor
    slots: torch.Tensor               # int64 [T]
    pairs: Optional[torch.Tensor]     # int32 [n, 2] copy-on-write pairs, or None
    q: torch.Tensor                   # [num_q_tokens, H, d]
    block_tables: torch.Tensor        # int32 [S, max_blocks]
    context_lens: torch.Tensor        # int32 [S]
    query_start_loc: Optional[torch.Tensor]
    max_q_len: int
    max_context_len: int
    out: torch.Tensor
    workspace: Optional[torch.Tensor]
    shared: Optional["SharedPrefix"] = None
    weights_workspace: Optional[torch.Tensor] = None   # accumulate_step's, from its first call on
    q_lens: Optional[Sequence[int]] = None   # query run of every sequence
    seqs: Optional[Sequence] = None          # their names
    rotary: Optional[Rotary] = None          # then write_step rotates q and key into these:
    positions: Optional[torch.Tensor] = None       # int32 [axes, T]
    q_rotated: Optional[torch.Tensor] = None
    key_rotated: Optional[torch.Tensor] = None
    prompt_start: Optional[torch.Tensor] = None    # int32 [S + 1]: whole prompts, attended as rows


def _queries(si) -> torch.Tensor:
    """The queries of a step that attention takes: rotated, where its write rotates them."""
    rotated = getattr(si, "q_rotated", None)
    return si.q if rotated is None else rotated


@dataclass
class SharedPrefix:
    """Fork groups of a step for read-once shared-prefix decode."""
    group_start: torch.Tensor         # int32 [G + 1] (device)
    prefix_len: torch.Tensor          # int32 [G] (device)
    group_start_host: np.ndarray
    prefix_len_host: np.ndarray
    max_group_q_len: int
    max_prefix_len: int
    workspace: torch.Tensor


@dataclass
class TokenWeights:
    """What attention has given every cached token of a batch of sequences (one
    row per sequence, in the order of `seqs`), by which tokens are evicted."""
    seqs: List
    scores: torch.Tensor              # fp32 [S, H_kv, width]
    positions: torch.Tensor           # int32 [S, H_kv, width], -1: in text order
    evicted: np.ndarray               # int64 [S]: tokens evicted so far
    settled: Optional[np.ndarray] = None   # int64 [S]: tokens the last eviction left, in no order

    def __post_init__(self):
        if self.settled is None:
            self.settled = np.zeros(len(self.seqs), np.int64)


class PagedKVCache:
    def __init__(self, num_blocks: int, num_kv_heads: int, head_dim: int, kv_dtype: str,
                 device="cuda", free_order: Optional[Sequence[int]] = None,
                 canary_blocks: int = 0, canary_byte: int = 0, head_scales=None):
        """head_scales: FP8 caches only, (k_scale, v_scale) per KV head (fp32,
        calibrated by the caller)."""
        self.num_blocks = num_blocks
        self.num_kv_heads = num_kv_heads
        self.head_dim = head_dim
        self.kv_dtype = kv_dtype
        self.device = torch.device(device)
        self.pool = Pool(num_blocks, BLOCK_SIZE, free_order)
        nb = num_blocks + canary_blocks
        shp = (nb, num_kv_heads, BLOCK_SIZE, head_dim)
        if kv_dtype == "int4":     # two elements to a byte
            shp = shp[:3] + (head_dim // 2,)
        self.k = torch.zeros(shp, dtype=KV_TORCH[kv_dtype], device=self.device)
        self.v = torch.zeros(shp, dtype=KV_TORCH[kv_dtype], device=self.device)
        self.k_scale = self.v_scale = self.k_zp = self.v_zp = None
        if kv_dtype in ("int8", "int4"):
            row = shp[:3] + ((head_dim // INT4_GROUP,) if kv_dtype == "int4" else ())
            self.k_scale = torch.zeros(row, dtype=torch.float32, device=self.device)
            self.v_scale = torch.zeros(row, dtype=torch.float32, device=self.device)
            self.k_zp = torch.zeros(row, dtype=torch.int8, device=self.device)
            self.v_zp = torch.zeros(row, dtype=torch.int8, device=self.device)
        if kv_dtype == "fp8":
            if head_scales is None:
                raise ValueError("an FP8 cache needs per-head scales (k_scale, v_scale)")
            ks, vs = head_scales
            self.k_scale = torch.as_tensor(np.asarray(ks, np.float32)).to(self.device)
            self.v_scale = torch.as_tensor(np.asarray(vs, np.float32)).to(self.device)
        if canary_blocks:
            for t in self.arrays():
                t[num_blocks:].view(torch.uint8).fill_(canary_byte)

    def arrays(self) -> List[torch.Tensor]:
        out = [self.k, self.v]
        if self.kv_dtype in ("int8", "int4"):
            out += [self.k_scale, self.v_scale, self.k_zp, self.v_zp]
        return out

    # -- host side of a phase: reserve slots, collect copy pairs --------------
    def reserve(self, ops, names: Dict) -> tuple:
        slots, pairs, ks, vs = [], [], [], []
        for op in ops:
            if hasattr(op, "parent"):
                names[op.child] = self.pool.seq_fork(names[op.parent])
            elif hasattr(op, "k"):
                sl, pair = self.pool.seq_append_slots(names[op.seq], int(op.k.shape[0]))
                if pair is not None:
                    pairs.append(pair)
                slots.append(sl)
                ks.append(op.k)
                vs.append(op.v)
            else:
                names[op.seq] = self.pool.seq_create()
        sl = np.concatenate(slots) if slots else np.zeros(0, np.int64)
        return sl, pairs, ks, vs

    # -- device side: copies first, then the append ------------------------------
    def write(self, slots: np.ndarray, pairs, ks, vs) -> None:
        if pairs:
            pr = torch.tensor(pairs, dtype=torch.int32, device=self.device)
            copy_blocks(self.k, self.v, pr, self.num_blocks, self.k_scale, self.v_scale,
                        self.k_zp, self.v_zp)
        if len(slots):
            key = torch.cat(ks).to(self.device)
            value = torch.cat(vs).to(self.device)
            sl = torch.from_numpy(np.ascontiguousarray(slots)).to(self.device)
            append_kv(key, value, self.k, self.v, sl, self.num_blocks, self.k_scale,
                      self.v_scale, self.k_zp, self.v_zp)

    def run_phase(self, ops, names: Dict) -> tuple:
        slots, pairs, ks, vs = self.reserve(ops, names)
        self.write(slots, pairs, ks, vs)
        return slots, pairs

    # -- decode step -------------------------------------------------------------
    def _check_positions(self, step_ops, names: Dict, rotary: Rotary, positions, reserve) -> None:
        """A step's positions lie within its table of angles: the cache would keep what its
        slots held before, and attention take rows that nothing was written to."""
        most, runs = rotary.cos_sin.shape[0], [int(op.k.shape[0]) for op in step_ops]
        if positions is None:
            end: Dict = {}
            for op, r in zip(step_ops, runs):
                s = names[op.seq]
                if s not in end:
                    end[s] = self.pool.seq_len(s) + self.pool.evicted.get(s, 0)
                end[s] += r if reserve else 0
                if r and end[s] > most:
                    raise ValueError(f"sequence {op.seq!r} reaches position {end[s] - 1}, the table "
                                     f"of angles has {most}")
            return
        at = tuple(np.shape(positions))
        if len(at) not in (1, 2) or at[-1] != sum(runs):
            raise ValueError(f"positions are {at}, the step has {sum(runs)} tokens")
        if not (torch.is_tensor(positions) and positions.is_cuda):
            p = np.asarray(positions)
            if p.size and (p.min() < 0 or p.max() >= most):
                raise ValueError(f"positions of {p.min()} to {p.max()}, the table of angles has {most}")

    def prepare_step(self, step_ops, names: Dict, q: torch.Tensor, out_dtype=None,
                     partition_size: int = 0, reserve: bool = True,
                     shared_prefix: bool = False, rotary: Optional[Rotary] = None,
                     positions=None, prompt: bool = False) -> StepInputs:
        """Reserve the step's slots (host) and build its device inputs. With
        shared_prefix, also the fork groups (adjacent sequences of the step
        holding the same prompt blocks), so that attend_step reads each
        group's shared blocks once.

        rotary: q and the keys of the operations are rotated by write_step on their way
        into the cache. positions: int [T] or [axes, T] of the step's tokens; without it a
        token's place in its sequence, evicted tokens counted. A position past the table is
        refused before anything is reserved (those of a device tensor are not looked at here:
        pa_rope_append_kv leaves their tokens out).

        prompt: the operations are whole prompts, each all the tokens of its sequence;
        attend_step then attends them from the rows themselves (the cache's type does not
        matter to it), and the output has the type of q. Other steps' is fp32 unless
        out_dtype says otherwise."""
        if prompt:
            if len({op.seq for op in step_ops}) < len(step_ops):
                raise ValueError("a sequence appears twice among the prompts")
            for op in step_ops:
                held = self.pool.seq_len(names[op.seq]) - (0 if reserve else int(op.k.shape[0]))
                if held:
                    raise ValueError(f"sequence {op.seq!r} holds {held} tokens before this prompt")
            if out_dtype not in (None, q.dtype) or partition_size or shared_prefix:
                raise ValueError("a prompt's output has the type of q; it has no partitions and "
                                 "no shared prefix")
        out_dtype = out_dtype or (q.dtype if prompt else torch.float32)
        if rotary is not None:
            self._check_positions(step_ops, names, rotary, positions, reserve)
        slots, pairs, ks, vs = self.reserve(step_ops, names) if reserve else (None, [], [], [])
        seqs = [names[op.seq] for op in step_ops]
        q_lens = [int(op.k.shape[0]) for op in step_ops]
        lens = [self.pool.seq_len(s) for s in seqs]
        max_blocks = max(1, max((L + BLOCK_SIZE - 1) // BLOCK_SIZE for L in lens))
        bt, cl = self.pool.block_tables(seqs, max_blocks)
        dev = self.device
        multi = max(q_lens) > 1
        qsl = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        nq = int(qsl[-1])
        if rotary is not None:
            if positions is None:
                positions = np.concatenate(
                    [L - r + self.pool.evicted.get(s, 0) + np.arange(r)
                     for s, L, r in zip(seqs, lens, q_lens)])
            positions = torch.as_tensor(positions, dtype=torch.int32).to(dev).contiguous()
        ws_bytes = (prompt_attention_workspace_size(q.shape[2], max(q_lens)) if prompt else
                    decode_workspace_size(len(seqs), nq, q.shape[1], self.num_kv_heads, q.shape[2],
                                          max(q_lens), max(lens), partition_size))
        shared = None
        if shared_prefix:
            gs, pl = self.pool.prefix_groups(seqs, q_lens)
            gq = [int(qsl[gs[g + 1]] - qsl[gs[g]]) for g in range(len(pl))]
            sp_bytes = decode_shared_prefix_workspace_size(
                len(seqs), nq, q.shape[1], self.num_kv_heads, q.shape[2], max(q_lens), max(lens),
                len(pl), max(gq), int(pl.max()), max_blocks)
            shared = SharedPrefix(
                group_start=torch.from_numpy(gs).to(dev), prefix_len=torch.from_numpy(pl).to(dev),
                group_start_host=gs, prefix_len_host=pl, max_group_q_len=max(gq),
                max_prefix_len=int(pl.max()),
                workspace=zeroed_workspace(sp_bytes, dev))
        key, q = torch.cat(ks).to(dev), q.to(dev).contiguous()
        return StepInputs(
            key=key, value=torch.cat(vs).to(dev),
            slots=torch.from_numpy(np.ascontiguousarray(slots)).to(dev),
            pairs=(torch.tensor(pairs, dtype=torch.int32, device=dev) if pairs else None),
            q=q,
            block_tables=torch.from_numpy(bt).to(dev),
            context_lens=torch.from_numpy(cl).to(dev),
            query_start_loc=torch.from_numpy(qsl).to(dev) if multi else None,
            max_q_len=max(q_lens), max_context_len=max(lens),
            out=torch.empty((nq, q.shape[1], q.shape[2]), dtype=out_dtype, device=dev),
            workspace=zeroed_workspace(ws_bytes, dev),
            shared=shared, q_lens=q_lens, seqs=[op.seq for op in step_ops],
            rotary=rotary, positions=None if rotary is None else positions,
            q_rotated=None if rotary is None else torch.empty_like(q),
            key_rotated=None if rotary is None else torch.empty_like(key),
            prompt_start=torch.from_numpy(qsl).to(dev) if prompt else None)

    def write_step(self, si: StepInputs) -> None:
        """The step's cache writes: copy-on-write block copies, then the append."""
        if si.pairs is not None:
            copy_blocks(self.k, self.v, si.pairs, self.num_blocks, self.k_scale,
                        self.v_scale, self.k_zp, self.v_zp)
        if si.rotary is not None:
            rope_append_kv(si.q_rotated, si.q, si.key, si.value, self.k, self.v, si.slots,
                           si.rotary.cos_sin, si.positions, self.num_blocks, self.k_scale,
                           self.v_scale, self.k_zp, self.v_zp, si.key_rotated,
                           si.rotary.interleaved, si.rotary.freq_axis)
            return
        append_kv(si.key, si.value, self.k, self.v, si.slots, self.num_blocks,
                  self.k_scale, self.v_scale, self.k_zp, self.v_zp)

    def attend_step(self, si: StepInputs, scale: float, partition_size: int = 0) -> torch.Tensor:
        """The step's attention over the cache (decode kernel + partial merge), or of whole
        prompts over their own rows. Rotated queries are those that write_step left."""
        if si.prompt_start is not None:
            key = si.key if si.key_rotated is None else si.key_rotated
            prompt_attention(si.out, _queries(si), key, si.value, si.prompt_start, si.max_q_len,
                             scale, si.workspace)
            return si.out
        if si.shared is not None:
            sp = si.shared
            decode_shared_prefix(si.out, _queries(si), self.k, self.v, si.block_tables, si.context_lens,
                                 si.max_context_len, scale, sp.group_start, sp.prefix_len,
                                 sp.max_group_q_len, sp.max_prefix_len, si.query_start_loc,
                                 si.max_q_len, self.num_blocks, sp.workspace)
            return si.out
        decode(si.out, _queries(si), self.k, self.v, si.block_tables, si.context_lens,
               si.max_context_len, scale, si.query_start_loc, si.max_q_len, self.num_blocks,
               self.k_scale, self.v_scale, self.k_zp, self.v_zp, partition_size,
               si.workspace)
        return si.out

    def step(self, si: StepInputs, scale: float, partition_size: int = 0,
             write: bool = True) -> torch.Tensor:
        """One decode step on device-resident inputs: copies, append, attend."""
        if write:
            self.write_step(si)
        return self.attend_step(si, scale, partition_size)

    # -- eviction by accumulated attention weight ---------------------------------
    def track_weights(self, seqs: Sequence, width: int, carry: Sequence[TokenWeights] = (),
                      parents: Optional[Dict] = None) -> TokenWeights:
        """Weights for `seqs` (caller-chosen names), up to `width` tokens each: of a batch
        whose sequences come and go, a new one when it changes. A sequence that one of
        `carry` tracks, or whose parent there (`parents`: a fork's name to its parent's)
        does, comes over with its weights and positions; the others start from none. A
        sequence that has lost tokens to an eviction has to come over; rows go by name,
        so a name given to a new sequence is not to be found in `carry`."""
        shape = (len(seqs), self.num_kv_heads, width)
        tw = TokenWeights(list(seqs), torch.zeros(shape, device=self.device),
                          torch.full(shape, -1, dtype=torch.int32, device=self.device),
                          np.zeros(len(seqs), np.int64))
        for i, name in enumerate(seqs):
            source = (parents or {}).get(name, name)
            old = next((t for t in carry if source in t.seqs), None)
            if old is None:
                continue
            j, n = old.seqs.index(source), min(width, old.scores.shape[2])
            tw.scores[i, :, :n] = old.scores[j, :, :n]
            tw.positions[i, :, :n] = old.positions[j, :, :n]
            tw.evicted[i], tw.settled[i] = old.evicted[j], old.settled[j]
        return tw

    def _tracked(self, tw: TokenWeights, names: Dict) -> List[int]:
        """The pool's ids of tw's sequences, whose evictions tw has to know of: a row that
        does not takes kept tokens for the first ones of the text."""
        ids = [names[s] for s in tw.seqs]
        if len(set(ids)) != len(ids):
            raise ValueError("a sequence appears twice")
        for s, i, n in zip(tw.seqs, ids, tw.evicted):
            if self.pool.evicted.get(i, 0) != n:
                raise ValueError(f"sequence {s!r} has lost {self.pool.evicted.get(i, 0)} tokens to "
                                 f"evictions, {n} in these weights: carry its row over "
                                 "(track_weights)")
        return ids

    def accumulate_step(self, si: StepInputs, tw: TokenWeights, scale: float,
                        accepted: Optional[Sequence[int]] = None) -> None:
        """Add the weights of the step's queries (rows of si and tw alike). The workspace
        is the step's own, so that a captured step keeps the one it was captured with.

        accepted: of a verify step, how many of every sequence's queries count, from the
        first on; the tokens of the others are those that truncate() takes back, before
        or after this call. Host numbers, so such a call is not captured. Without it
        every query counts, and what rejected ones gave stays in the sums."""
        if si.seqs is not None and list(si.seqs) != tw.seqs:
            raise ValueError(f"the step is of {list(si.seqs)}, the weights of {tw.seqs}")
        q, lens, start = _queries(si), si.context_lens, si.query_start_loc
        if accepted is not None:
            runs = np.asarray(si.q_lens, np.int64)
            acc = np.asarray(accepted, np.int64)
            if acc.shape != runs.shape or (acc < 0).any() or (acc > runs).any():
                raise ValueError(f"accepted {acc.tolist()} of query runs {runs.tolist()}")
            first = np.cumsum(runs) - runs
            rows = np.concatenate([f + np.arange(a) for f, a in zip(first, acc)])
            # a call has at least as many queries as sequences: those behind the last run add nothing
            rows = np.append(rows, np.zeros(max(0, len(runs) - len(rows)), np.int64))

            def to(a, dtype):
                return torch.from_numpy(np.ascontiguousarray(a, dtype)).to(self.device)

            q = q[to(rows, np.int64)]
            lens = lens - to(runs - acc, np.int32)
            start = to(np.append(0, np.cumsum(acc)), np.int32)
        n = accumulate_weights_workspace_size(si.context_lens.shape[0], si.q.shape[0],
                                              si.q.shape[1], self.num_kv_heads, self.head_dim,
                                              si.max_q_len, si.max_context_len)
        if si.weights_workspace is None or si.weights_workspace.numel() < n:
            si.weights_workspace = torch.empty(n, dtype=torch.uint8, device=self.device)
        accumulate_weights(tw.scores, tw.scores, q, self.k, si.block_tables, lens,
                           si.max_context_len, scale, start, si.max_q_len,
                           self.num_blocks, self.k_scale, self.k_zp, si.weights_workspace)

    def truncate(self, tw: TokenWeights, names: Dict, lens) -> None:
        """Take back the tokens of tw's sequences past the first `lens` (an int, or one per
        sequence; a shorter sequence stays as it is), as rejected draft tokens, and the
        weights they received: the next tokens in their slots start from none. Tokens that
        an eviction left stand in no order and cannot be cut by their slots."""
        ids = self._tracked(tw, names)
        now = np.array([self.pool.seq_len(i) for i in ids], np.int64)
        new = np.minimum(np.broadcast_to(np.asarray(lens, np.int64), now.shape), now)
        if (new < 0).any():
            raise ValueError("a length is negative")
        for s, n, old, kept in zip(tw.seqs, new, now, tw.settled):
            if n < old and n < kept:
                raise ValueError(f"sequence {s!r}: its first {kept} tokens are what an eviction "
                                 f"left, which {n} would cut")
        if not (new < now).any():
            return
        for i, n in zip(ids, new):
            self.pool.seq_truncate(i, int(n))
        past = (torch.arange(tw.scores.shape[2], device=tw.scores.device) >=
                torch.from_numpy(new).to(tw.scores.device)[:, None, None])
        tw.scores.masked_fill_(past, 0)
        tw.positions.masked_fill_(past, -1)

    def evict(self, tw: TokenWeights, names: Dict, keep, num_sinks: int = 0,
              num_recent: int = 0) -> None:
        """Bring every sequence of tw down to `keep` tokens (an int, or one per
        sequence; a shorter sequence stays as it is): blocks that will be
        written become its own (copied where shared), the kept tokens are chosen
        per KV head, their rows moved, and the freed blocks given back. Where the
        pool cannot cover the copies it raises, and no token has gone."""
        ids = self._tracked(tw, names)
        lens = np.array([self.pool.seq_len(i) for i in ids], np.int64)
        kept = np.minimum(np.broadcast_to(np.asarray(keep, np.int64), lens.shape), lens)
        if (kept < 0).any():
            raise ValueError("keep is negative")
        if lens.size and lens.max() > tw.scores.shape[2]:
            raise ValueError(f"a sequence holds {lens.max()} tokens, its weights {tw.scores.shape[2]}")
        if not (kept < lens).any():
            return
        for i, n, L in zip(ids, kept, lens):
            if n < L:
                # copied at once: a later sequence's error leaves a consistent cache
                pairs = self.pool.seq_make_private(i, int(n))
                if len(pairs):
                    copy_blocks(self.k, self.v, torch.from_numpy(pairs).to(self.device),
                                self.num_blocks, self.k_scale, self.v_scale, self.k_zp, self.v_zp)
        width = int(lens.max())
        bt, cl = self.pool.block_tables(ids, -(-width // BLOCK_SIZE))
        dev = self.device

        def to(a):
            return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)

        shape = tw.scores.shape[:2]
        moves = torch.empty((*shape, max(1, width // 2), 2), dtype=torch.int32, device=dev)
        counts = torch.empty(shape, dtype=torch.int32, device=dev)
        lens_d = to(cl)
        evict_select(moves, counts, tw.scores, tw.positions, tw.scores, tw.positions, lens_d,
                     to(kept), to(lens + tw.evicted), width, num_sinks, num_recent)
        move_tokens(self.k, self.v, to(bt), lens_d, moves, counts, width, self.num_blocks,
                    self.k_scale, self.v_scale, self.k_zp, self.v_zp)
        for i, n in zip(ids, kept):
            self.pool.seq_truncate(i, int(n))
        tw.evicted += lens - kept
        self.pool.evicted.update((i, int(n)) for i, n in zip(ids, tw.evicted) if n)
        tw.settled = np.where(kept < lens, kept, tw.settled)

    def capture(self, fn, *args) -> "torch.cuda.CUDAGraph":
        """Record fn(*args) (e.g. write_step or attend_step) in a CUDA graph;
        graph.replay() then runs the same kernels on the same buffers with no
        per-launch host work. fn runs once eagerly first, so the library's
        one-time set-up (tensor maps, kernel attributes) happens outside the
        capture."""
        fn(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn(*args)
        torch.cuda.synchronize()
        return g
