"""One attention layer's paged KV cache on one GPU.

The pool is allocated once as two device arrays [num_blocks, Hkv, 16, D]
("The inference server": the KV cache is one arena allocated at start-up,
managed by block tables, with no allocator on the hot path). The C++ block
manager owns the tables; a decode step is host bookkeeping (slots and
copy-on-write pairs from pkv_bm_prepare_append, cs2680 Lecture 10, §10.5's
"allocate blocks to grow") followed by three launches on one stream: block
copy, append, attention.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import numpy as np
import torch

from . import _native as nat


def bf16_from_bits(bits: np.ndarray) -> torch.Tensor:
    """uint16 bf16 bit patterns -> CPU bf16 tensor sharing no arithmetic."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)


def bits_from_bf16(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def shared_prefix_groups(tables, context_lens, block_tokens: int = nat.BLOCK_TOKENS, min_members: int = 2):
    """Groups of a batch's sequences that share leading blocks, for cascade
    attention: sequences whose tables start with the same block form a group
    (of at least min_members); its shared length is the longest table prefix
    all members agree on, limited to the complete blocks of the shortest
    member (a shared tile must be whole for every sharer). Host arithmetic on
    the batch's block tables; returns [(member indices, shared blocks)]."""
    tables = np.asarray(tables)
    ctx = np.asarray(context_lens, dtype=np.int64)
    by_first = {}
    for s in range(len(ctx)):
        if ctx[s] >= block_tokens:
            by_first.setdefault(int(tables[s, 0]), []).append(s)
    groups = []
    for members in by_first.values():
        if len(members) < min_members:
            continue
        limit = int(min(ctx[m] // block_tokens for m in members))
        rows = tables[members, :limit]
        agree = np.all(rows == rows[0], axis=0)
        shared = limit if agree.all() else int(np.argmin(agree))
        if shared >= 1:
            groups.append((members, shared))
    return groups


# Below this many K/V bytes saved, the cascade's extra launches cost more than
# the shared reads they avoid (measured: a 7-request group sharing 128 blocks,
# 59 MB saved, ran slower than the plain kernel; 16 prompts x 8 samples,
# 1.06 GB saved, ran 2.3x faster).
CASCADE_MIN_SAVED_BYTES = 128 << 20


def cascade_saved_bytes(groups, num_kv_heads: int, block_tokens: int = nat.BLOCK_TOKENS, head_dim: int = 128) -> int:
    """K and V bytes cascade attention does not read: every sharer but one of
    each group skips the group's shared blocks."""
    per_block = num_kv_heads * block_tokens * head_dim * 2 * 2
    return sum((len(m) - 1) * sh * per_block for m, sh in groups)


@dataclass
class StepBuffers:
    """Device inputs and output of one decode step (shapes fixed per batch)."""
    seq_ids: list
    slots: torch.Tensor       # int64 [B]
    pairs: torch.Tensor       # int32 [n, 2]
    tables: torch.Tensor      # int32 [B, W]
    ctx: torch.Tensor         # int32 [B]
    q: torch.Tensor           # bf16 [B, Hq, D]
    k: torch.Tensor           # bf16 [B, Hkv, D]
    v: torch.Tensor           # bf16 [B, Hkv, D]
    out: torch.Tensor         # bf16 [B, Hq, D]
    workspace: nat.AttentionWorkspace

    @property
    def num_pairs(self) -> int:
        return int(self.pairs.shape[0])


@dataclass
class RopeSpec:
    """How a layer's queries and keys enter the cache: rotation by a table of
    rope_table() and the heads' norm weights (None: no norm)."""
    cos_sin: torch.Tensor
    q_weight: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None
    eps: float = 1e-6
    interleaved: bool = False


@dataclass
class Int4Pages:
    """The pages of a batch's contexts in a 4-bit cache, and where they lie once they
    are loaded as bf16 pages, each page once."""
    pairs: torch.Tensor       # int32 [n, 2]: block, place
    tables: torch.Tensor      # int32 [B, W] of places


@dataclass
class PromptBuffers:
    """Device inputs of one prefill call: packed rows of several sequences."""
    seq_ids: list
    counts: list
    positions: torch.Tensor   # int32 [T]
    tables: torch.Tensor      # int32 [B, W]
    ctx: torch.Tensor         # int32 [B], the chunk included
    starts: torch.Tensor      # int32 [B + 1]
    slots: torch.Tensor       # int64 [T]
    pages: Int4Pages | None = None


@dataclass
class DraftBuffers:
    """Device inputs of one verification step of drafted trees."""
    seq_ids: list
    counts: list
    positions: torch.Tensor   # int32 [T]
    tables: torch.Tensor      # int32 [B, W]
    ctx: torch.Tensor         # int32 [B], the drafts not included
    starts: torch.Tensor      # int32 [B + 1]
    masks: torch.Tensor       # int64 [T]
    slots: torch.Tensor       # int64 [T], all -1: nothing is appended yet
    held: list                # the sequences' context lengths
    parents: list             # the sequences' trees
    pages: Int4Pages | None = None


class PagedKVEngine:
    """cache_bits 16: the pools k_cache and v_cache hold bf16. cache_bits 4: `cache`
    (an Int4Cache) holds keys and values quantised in groups of group_dims; what
    is attended, by decode steps, prompts and drafts alike, is what it holds."""

    def __init__(self, num_blocks: int, num_q_heads: int, num_kv_heads: int, head_dim: int = 128,
                 device="cuda", free_order=None, block_tokens: int = nat.BLOCK_TOKENS, incremental: bool = False,
                 watermark: int = 0, prefix_cache: bool = False, cache_bits: int = 16, group_dims: int = 64):
        if cache_bits not in (4, 16):
            raise ValueError("cache_bits is 4 or 16")
        if cache_bits == 4 and head_dim != nat.HEAD_DIM:
            raise ValueError(f"a 4-bit cache has heads of {nat.HEAD_DIM} values")
        self.num_blocks, self.num_q_heads, self.num_kv_heads, self.head_dim = (
            num_blocks, num_q_heads, num_kv_heads, head_dim)
        self.block_tokens = block_tokens
        self.device = torch.device(device)
        self.k_cache = self.v_cache = self.cache = None
        if cache_bits == 4:
            self.cache = nat.Int4Cache(num_blocks, num_kv_heads, block_tokens, group_dims, device=self.device)
        else:
            shape = (num_blocks, num_kv_heads, block_tokens, head_dim)
            self.k_cache = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            self.v_cache = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        self.bm = nat.BlockManager(num_blocks, block_tokens, free_order, incremental=incremental,
                                   watermark=watermark, prefix_cache=prefix_cache)
        self.error = nat.new_error_word(self.device)

    # ---- pool content ----------------------------------------------------
    def load_pool(self, k_bits: np.ndarray, v_bits: np.ndarray, lo: int = 0) -> None:
        n = k_bits.shape[0]
        if self.cache is not None:
            rows = [bf16_from_bits(b).to(self.device).transpose(1, 2).reshape(n * self.block_tokens, self.num_kv_heads, -1)
                    for b in (k_bits, v_bits)]
            first = lo * self.block_tokens
            self._write(*rows, torch.arange(first, first + n * self.block_tokens, device=self.device))
            return
        self.k_cache[lo : lo + n].copy_(bf16_from_bits(k_bits))
        self.v_cache[lo : lo + n].copy_(bf16_from_bits(v_bits))

    def load_workload_pool(self, w, chunk_blocks: int = 4096) -> None:
        for lo in range(0, w.pool_blocks, chunk_blocks):
            hi = min(w.pool_blocks, lo + chunk_blocks)
            self.load_pool(w.pool_blocks_range("k", lo, hi), w.pool_blocks_range("v", lo, hi), lo)

    # ---- host bookkeeping + device launches ---------------------------------
    def _side(self, stream) -> torch.cuda.Stream:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        return stream

    def _on(self, stream):
        """A context in which `stream` (default: the current one) is current, so
        that what is allocated inside belongs to it."""
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(self._side(stream))

    def _keep(self, stream, *inputs) -> None:
        """The memory of inputs that the caller made on another stream is not given
        out anew before `stream` is done with them."""
        if stream is not None:
            for t in inputs:
                if t.is_cuda:  # others are refused by the call itself
                    t.record_stream(self._side(stream))

    def _write(self, k, v, slots, stream=None) -> None:
        if self.cache is not None:
            nat.append_int4(k, v, slots, self.cache, self.error, stream)
        else:
            nat.append(k, v, slots, self.k_cache, self.v_cache, self.error, stream)

    def _copy(self, pairs, stream=None) -> None:
        if self.cache is not None:
            nat.block_copy_int4(self.cache, pairs, self.error, stream)
        else:
            nat.block_copy(self.k_cache, self.v_cache, pairs, self.error, stream)

    def append_tokens(self, seq_ids, k: torch.Tensor, v: torch.Tensor, stream=None):
        """Append one token per sequence (k, v: [B, Hkv, D] bf16 on device);
        returns (slots, pairs) as the block manager decided them."""
        slots, pairs = self.bm.prepare_append(list(seq_ids))
        with self._on(stream):
            if pairs:
                pt = torch.tensor(pairs, dtype=torch.int32).to(self.device, non_blocking=True)
                self._copy(pt)
            st = torch.tensor(slots, dtype=torch.int64).to(self.device, non_blocking=True)
            self._write(k, v, st)
        self._keep(stream, k, v)
        return slots, pairs

    def write_positions(self, seq_id: int, first: int, k: torch.Tensor, v: torch.Tensor, stream=None):
        """Write the KV of token positions [first, first + n) of one sequence
        (k, v: [n, Hkv, D] bf16 on device) -- a prefill, or the recompute of a
        resumed sequence -- with the append kernel; returns the slots."""
        slots = self.bm.slots(seq_id, first, int(k.shape[0]))
        with self._on(stream):
            st = torch.tensor(slots, dtype=torch.int64).to(self.device, non_blocking=True)
            self._write(k, v, st)
        self._keep(stream, k, v)
        self._wrote(seq_id, first, len(slots))
        return slots

    # ---- prompts and drafted tokens -------------------------------------------
    def prepare_prefill(self, seq_ids, counts, first=None) -> PromptBuffers:
        """Host bookkeeping of a prefill call: sequence seq_ids[i] brings counts[i]
        tokens of its prompt, from position first[i] on. Without first they are
        its last ones: the whole prompt, the rest of one, or a token that a decode
        step's append made room for. Prompt tokens before them have to be in the
        cache or on their way (an earlier chunk's, write_positions', a cached or
        shared prefix's): a chunk that leaves some out needs first (ValueError).
        The slots lie in the pages that admission reserved."""
        seq_ids, counts = list(seq_ids), [int(c) for c in counts]
        if first is None:
            first = [self.bm.context_len(s) - c for s, c in zip(seq_ids, counts)]
            for s, f, c in zip(seq_ids, first, counts):
                if c and f > self._known(s):
                    raise ValueError(f"a chunk of {c} of sequence {s}'s {f + c} tokens needs its first position")
        if len(seq_ids) != len(counts) or len(first) != len(counts):
            raise ValueError("one count and one first position per sequence")
        for s, f, c in zip(seq_ids, first, counts):
            if f < 0 or c < 0 or f + c > self.bm.context_len(s):
                raise ValueError(f"positions {f} to {f + c} leave sequence {s}'s {self.bm.context_len(s)} tokens")
        slots, positions = [], []
        for s, f, c in zip(seq_ids, first, counts):
            slots += self.bm.slots(s, f, c) if c else []
            self._wrote(s, f, c)
            positions += range(f, f + c)
        held = [f + c for f, c in zip(first, counts)]
        return PromptBuffers(*self._rows(seq_ids, counts, held, positions),
                             slots=torch.tensor(slots, dtype=torch.int64).to(self.device), pages=self._pages(seq_ids, held))

    def _known(self, seq_id) -> int:
        """A sequence's tokens, from the first on, that are in the cache or on their
        way: those written, those in blocks that other sequences hold too, and all
        behind the prompt."""
        table = self.bm.table(seq_id)
        shared = next((i for i, b in enumerate(table) if self.bm.refcount(b) < 2), len(table))
        known = max(self.bm.written[seq_id], shared * self.block_tokens)
        return self.bm.context_len(seq_id) if known >= self.bm.prompt[seq_id] else known

    def _wrote(self, seq_id, first: int, n: int) -> None:
        if n and self.bm.written[seq_id] < first + n and first <= self._known(seq_id):
            self.bm.written[seq_id] = first + n

    def _rows(self, seq_ids, counts, context_lens, positions):
        if not seq_ids:
            raise ValueError("at least one sequence")
        tables, _ = self.bm.batch_tables(seq_ids, max(1, max(len(self.bm.table(s)) for s in seq_ids)))
        starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        ints = lambda x: torch.tensor(x, dtype=torch.int32).to(self.device)
        return seq_ids, counts, ints(positions), tables.to(self.device), ints(context_lens), torch.from_numpy(starts).to(self.device)

    def _pages(self, seq_ids, context_lens) -> Int4Pages | None:
        if self.cache is None:
            return None
        rows = [self.bm.table(s)[: -(-c // self.block_tokens)] for s, c in zip(seq_ids, context_lens)]
        place = {b: i for i, b in enumerate(dict.fromkeys(b for row in rows for b in row))}
        tables = torch.full((len(rows), max(1, max(len(row) for row in rows))), -1, dtype=torch.int32)
        for i, row in enumerate(rows):
            tables[i, : len(row)] = torch.tensor([place[b] for b in row], dtype=torch.int32)
        pairs = torch.tensor(list(place.items()), dtype=torch.int32).reshape(-1, 2)
        return Int4Pages(pairs.to(self.device), tables.to(self.device))

    def _room(self, pages: Int4Pages):
        """bf16 pools for the pages."""
        shape = (max(1, pages.pairs.shape[0]), self.num_kv_heads, self.block_tokens, self.head_dim)
        return [torch.empty(shape, dtype=torch.bfloat16, device=self.device) for _ in range(2)]

    def _turn(self, rope, q, k, v, positions, pools):
        """Normed, rotated queries and keys, nothing written to the pools."""
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        nowhere = torch.full((k.shape[0],), -1, dtype=torch.int64, device=k.device)
        q = nat.qk_norm_rope_append(q, k, v, rope.cos_sin, positions, nowhere, *pools, q_weight=rope.q_weight,
                                    k_weight=rope.k_weight, eps=rope.eps, interleaved=rope.interleaved, k_out=k_out,
                                    device_error=self.error)
        return q, k_out

    def run_prefill(self, pb: PromptBuffers, q, k, v, scale: float, workspace, rope=None, out=None, stream=None):
        """The device part: the chunk's keys and values into the cache, then
        causal attention of its rows. q [T, Hq, D], k, v [T, Hkv, D] (bf16 on the
        device), packed in pb's order."""
        self._keep(stream, q, k, v, pb.positions, pb.tables, pb.ctx, pb.starts, pb.slots)
        if self.cache is not None:
            return self._run_prefill_int4(pb, q, k, v, scale, workspace, rope, out, stream)
        with self._on(stream):
            if rope is None:
                nat.append(k, v, pb.slots, self.k_cache, self.v_cache, self.error)
            else:
                q = nat.qk_norm_rope_append(q, k, v, rope.cos_sin, pb.positions, pb.slots, self.k_cache, self.v_cache,
                                            q_weight=rope.q_weight, k_weight=rope.k_weight, eps=rope.eps,
                                            interleaved=rope.interleaved, device_error=self.error)
            return nat.attn_prefill(q, self.k_cache, self.v_cache, pb.tables, pb.ctx, pb.starts, scale, out=out,
                                    workspace=workspace)

    def _run_prefill_int4(self, pb, q, k, v, scale, workspace, rope, out, stream):
        """The chunk goes into the 4-bit cache, then the pages of its contexts, the
        chunk's own among them, come back as bf16 pages for the attention."""
        self._keep(stream, pb.pages.pairs, pb.pages.tables)
        with self._on(stream):
            pools = self._room(pb.pages)
            if rope is not None:
                q, k = self._turn(rope, q, k, v, pb.positions, pools)
            nat.append_int4(k, v, pb.slots, self.cache, self.error)
            nat.load_int4(self.cache, pb.pages.pairs, *pools, self.error)
            return nat.attn_prefill(q, *pools, pb.pages.tables, pb.ctx, pb.starts, scale, out=out, workspace=workspace)

    def prepare_drafts(self, seq_ids, parents) -> DraftBuffers:
        """Host bookkeeping of a verification step: sequence seq_ids[i] has the
        drafted tree parents[i] (see tree_masks()). A draft's position follows
        its parent's, or the context. Nothing is reserved or written."""
        seq_ids, parents = list(seq_ids), [list(p) for p in parents]
        ctx = [self.bm.context_len(s) for s in seq_ids]
        masks, positions = [], []
        for c, tree in zip(ctx, parents):
            masks += nat.tree_masks(tree)
            depth: list[int] = []
            for p in tree:
                depth.append(depth[p] + 1 if p >= 0 else 0)
            positions += [c + d for d in depth]
        rows = self._rows(seq_ids, [len(p) for p in parents], ctx, positions)
        return DraftBuffers(*rows, masks=torch.tensor(masks, dtype=torch.int64).to(self.device),
                            slots=torch.full((len(masks),), -1, dtype=torch.int64).to(self.device), held=ctx,
                            parents=parents, pages=self._pages(seq_ids, ctx))

    def run_drafts(self, db: DraftBuffers, q, k, v, scale: float, workspace, rope=None, out=None, stream=None):
        """The device part: (attention of the drafts, their keys as the cache would
        hold them); the cache stays as it was."""
        self._keep(stream, q, k, v, db.positions, db.tables, db.ctx, db.starts, db.masks, db.slots)
        if self.cache is not None:
            return self._run_drafts_int4(db, q, k, v, scale, workspace, rope, out, stream)
        with self._on(stream):
            if rope is not None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
                q = nat.qk_norm_rope_append(q, k, v, rope.cos_sin, db.positions, db.slots, self.k_cache, self.v_cache,
                                            q_weight=rope.q_weight, k_weight=rope.k_weight, eps=rope.eps,
                                            interleaved=rope.interleaved, k_out=k_out, device_error=self.error)
                k = k_out
            out = nat.attn_tree(q, k, v.contiguous(), db.masks, self.k_cache, self.v_cache, db.tables, db.ctx, db.starts,
                                scale, out=out, workspace=workspace)
        return out, k

    def _run_drafts_int4(self, db, q, k, v, scale, workspace, rope, out, stream):
        self._keep(stream, db.pages.pairs, db.pages.tables)
        with self._on(stream):
            pools = self._room(db.pages)
            if rope is not None:
                q, k = self._turn(rope, q, k, v, db.positions, pools)
            nat.load_int4(self.cache, db.pages.pairs, *pools, self.error)
            out = nat.attn_tree(q, k, v.contiguous(), db.masks, *pools, db.pages.tables, db.ctx, db.starts, scale, out=out,
                                workspace=workspace)
        return out, k

    def accept_drafts(self, db: DraftBuffers, paths, k, v, stream=None):
        """Append the accepted drafts, paths[i] = the chosen drafts of sequence i in
        order: the first follows the context, each other one the draft before it
        (their keys are rotated for those positions). k as run_drafts returned it.
        Returns the slots in draft order, -1 for the drafts that were not
        accepted. Where the manager refuses a token (PoolExhausted,
        ReservationExceeded), the drafts before it are appended all the same and
        the error is raised. A sequence whose context has grown since
        prepare_drafts takes no drafts (ValueError)."""
        paths = [[int(x) for x in p] for p in paths]
        if len(paths) != len(db.counts) or any(len(set(p)) != len(p) or any(not 0 <= x < n for x in p)
                                               for p, n in zip(paths, db.counts)):
            raise ValueError("one path per sequence, of different drafts of its own")
        if any(tree[x] != before for p, tree in zip(paths, db.parents) for before, x in zip([-1] + p, p)):
            raise ValueError("a path's first draft follows the context, and each other one's parent is the draft before it")
        grows = [i for i, p in enumerate(paths) if p]
        if len({db.seq_ids[i] for i in grows}) != len(grows) or any(
                self.bm.context_len(db.seq_ids[i]) != db.held[i] for i in grows):
            raise ValueError("a sequence takes one path, and only while its context is the one the drafts follow")
        starts = np.concatenate([[0], np.cumsum(db.counts)])
        slots = np.full(int(starts[-1]), -1, np.int64)
        pairs, refused = [], None
        for d in range(max((len(p) for p in paths), default=0)):
            rows = [i for i, p in enumerate(paths) if len(p) > d]
            try:
                got, cow = self.bm.prepare_append([db.seq_ids[i] for i in rows])
            except nat.PkvError as e:
                refused = e
                break
            pairs += cow
            for i, slot in zip(rows, got):
                slots[starts[i] + paths[i][d]] = slot
        self._keep(stream, k, v)
        with self._on(stream):
            if pairs:
                self._copy(torch.tensor(pairs, dtype=torch.int32).to(self.device))
            self._write(k, v.contiguous(), torch.from_numpy(slots).to(self.device))
        if refused is not None:
            raise refused
        return slots.tolist()

    def reorder(self, seq_ids, parents) -> None:
        """Sequence seq_ids[i] goes on as seq_ids[parents[i]] is now, as beam search
        asks after each selection: pages are shared by reference, and copied where
        prepare_step or append_tokens finds the next token in a shared one."""
        self.bm.reorder(seq_ids, parents)

    def replay_events(self, w, with_content: bool = True):
        """Apply a workload's admit / fork / history events; history appends
        write the workload's history K/V when with_content is set."""
        history = []
        for ei, ev in enumerate(w.events):
            if ev[0] == "admit":
                self.bm.admit(ev[1], ev[2], ev[3], ev[4])
            elif ev[0] == "fork":
                self.bm.fork(ev[1], ev[2])
            elif ev[0] == "history":
                counts = ev[1]
                ids = sorted(counts)
                for t in range(max(counts.values()) if counts else 0):
                    batch = [s for s in ids if counts[s] > t]
                    if with_content:
                        kb, vb = w.history_inputs(ei, t, len(batch))
                        k = bf16_from_bits(kb).to(self.device)
                        v = bf16_from_bits(vb).to(self.device)
                        slots, pairs = self.append_tokens(batch, k, v)
                    else:
                        slots, pairs = self.bm.prepare_append(batch)
                    history.append((batch, slots, pairs))
            else:
                raise ValueError(f"unknown event {ev[0]}")
        return history

    def prepare_step(self, seq_ids, q_bits, k_bits, v_bits, width: int | None = None) -> StepBuffers:
        """Host bookkeeping of one decode step (each sequence appends one
        token) and its device inputs; the step itself is run_step."""
        seq_ids = list(seq_ids)
        slots, pairs = self.bm.prepare_append(seq_ids)
        if width is None:
            width = max(len(self.bm.table(s)) for s in seq_ids)
        tables, ctx = self.bm.batch_tables(seq_ids, width)
        dev = self.device
        q = bf16_from_bits(q_bits).to(dev)
        return StepBuffers(
            seq_ids=seq_ids,
            slots=torch.tensor(slots, dtype=torch.int64).to(dev),
            pairs=torch.tensor(pairs, dtype=torch.int32).reshape(-1, 2).to(dev),
            tables=tables.to(dev), ctx=ctx.to(dev), q=q,
            k=bf16_from_bits(k_bits).to(dev), v=bf16_from_bits(v_bits).to(dev),
            out=torch.empty_like(q),
            workspace=nat.AttentionWorkspace(len(seq_ids), self.num_kv_heads, device=dev, int4=self.cache is not None))

    def run_step(self, sb: StepBuffers, scale: float, num_ctas: int = 0, stream=None) -> torch.Tensor:
        """The device part of a decode step -- copy-on-write copies, append,
        attention -- as one library call (separate calls for block sizes
        other than 16 and for a 4-bit cache). Idempotent for fixed inputs."""
        if self.cache is not None or self.block_tokens != nat.BLOCK_TOKENS:
            return self.run_step_separate(sb, scale, num_ctas, stream)
        return nat.decode_step(sb.q, sb.k, sb.v, sb.slots, sb.pairs, self.k_cache, self.v_cache, sb.tables,
                               sb.ctx, scale, sb.out, sb.workspace, self.error, num_ctas, stream)

    def run_step_separate(self, sb: StepBuffers, scale: float, num_ctas: int = 0, stream=None) -> torch.Tensor:
        """The same step as three separate library calls."""
        if sb.num_pairs:
            self._copy(sb.pairs, stream)
        self._write(sb.k, sb.v, sb.slots, stream)
        if self.cache is not None:
            return nat.attn_decode_int4(sb.q, self.cache, sb.tables, sb.ctx, scale, sb.out, sb.workspace, num_ctas, stream)
        nat.attn_decode(sb.q, self.k_cache, self.v_cache, sb.tables, sb.ctx, scale, sb.out,
                        sb.workspace, num_ctas, stream)
        return sb.out

    def cascade_for(self, sb: StepBuffers, min_saved_bytes: int = CASCADE_MIN_SAVED_BYTES):
        """A cascade plan for the step's batch when its shared prefixes save
        enough reads to pay for the extra launches, else None (as for a 4-bit
        cache, whose shared pages are read by each sequence)."""
        if self.cache is not None or self.block_tokens != nat.BLOCK_TOKENS:
            return None
        groups = shared_prefix_groups(sb.tables.cpu().numpy(), sb.ctx.cpu().numpy())
        if not groups or cascade_saved_bytes(groups, self.num_kv_heads, head_dim=self.head_dim) < min_saved_bytes:
            return None
        return nat.Cascade(len(sb.seq_ids), self.num_q_heads, self.num_kv_heads, groups, device=self.device)

    def run_step_cascade(self, sb: StepBuffers, scale: float, cascade, stream=None) -> torch.Tensor:
        """run_step with the attention through a cascade plan (copy-on-write
        copies and the append first, as in run_step)."""
        if self.cache is not None:
            raise ValueError("cascade attention reads a bf16 cache")
        if sb.num_pairs:
            nat.block_copy(self.k_cache, self.v_cache, sb.pairs, self.error, stream)
        nat.append(sb.k, sb.v, sb.slots, self.k_cache, self.v_cache, self.error, stream)
        return cascade.decode(sb.q, self.k_cache, self.v_cache, sb.tables, sb.ctx, scale, sb.out, stream)

    def read_errors(self, sb: StepBuffers | None = None) -> int:
        e = nat.read_device_error(self.error)
        if sb is not None:
            e |= sb.workspace.read_error()
        return e


class HostStep:
    """A decode step whose inputs and output live in host memory: one pinned
    packed input buffer (laid out by pkv_step_layout), its device staging
    buffer, and pinned output rows. run() is one pkv_decode_step_host call:
    a staging kernel reads the inputs across the host link, the step's
    kernels run, and the attention writes the output rows to host memory."""

    _DTYPES = {"q": torch.bfloat16, "k_new": torch.bfloat16, "v_new": torch.bfloat16, "slot_mapping": torch.int64,
               "block_tables": torch.int32, "context_lens": torch.int32, "src_dst_pairs": torch.int32}

    def __init__(self, eng: PagedKVEngine, num_seqs: int, width: int, max_pairs: int = 0):
        if eng.cache is not None or eng.block_tokens != nat.BLOCK_TOKENS:
            raise ValueError("host-buffer steps use a bf16 cache of 16-token blocks")
        self.eng, self.num_seqs, self.width, self.max_pairs = eng, num_seqs, width, max_pairs
        hq, hkv, d = eng.num_q_heads, eng.num_kv_heads, eng.head_dim
        self.layout = nat.step_layout(num_seqs, hq, hkv, d, width, max_pairs)
        self.shapes = {"q": (num_seqs, hq, d), "k_new": (num_seqs, hkv, d), "v_new": (num_seqs, hkv, d),
                       "slot_mapping": (num_seqs,), "block_tables": (num_seqs, width),
                       "context_lens": (num_seqs,), "src_dst_pairs": (max_pairs, 2)}
        nbytes = self.layout["bytes"]
        self.host = torch.zeros(nbytes, dtype=torch.uint8).pin_memory()
        buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=eng.device)
        off = (-buf.data_ptr()) % 256
        self._staging_buf, self.staging = buf, buf[off: off + nbytes]
        self.out_dev = torch.empty((num_seqs, hq, d), dtype=torch.bfloat16, device=eng.device)
        self.out_host = torch.empty((num_seqs, hq, d), dtype=torch.bfloat16).pin_memory()
        self.workspace = nat.AttentionWorkspace(num_seqs, hkv, device=eng.device)
        self.num_pairs = 0

    def field(self, name: str, rows: int | None = None) -> torch.Tensor:
        """Typed view of one input inside the pinned packed buffer."""
        shape = list(self.shapes[name])
        if rows is not None:
            shape[0] = rows
        dt = self._DTYPES[name]
        n = int(np.prod(shape)) * torch.tensor([], dtype=dt).element_size()
        off = self.layout[name]
        return self.host[off: off + n].view(dt).view(shape)

    def pack(self, q, k, v, slots, tables, ctx, pairs=None) -> int:
        """Copy a step's inputs (CPU tensors) into the packed buffer; returns
        its size in bytes for this number of pairs."""
        self.field("q").copy_(q)
        self.field("k_new").copy_(k)
        self.field("v_new").copy_(v)
        self.field("slot_mapping").copy_(torch.as_tensor(slots, dtype=torch.int64))
        self.field("block_tables").copy_(tables)
        self.field("context_lens").copy_(ctx)
        n = 0 if pairs is None else int(len(pairs))
        if n > self.max_pairs:
            raise ValueError(f"{n} copy pairs exceed the buffer's {self.max_pairs}")
        if n:
            self.field("src_dst_pairs", n).copy_(torch.as_tensor(pairs, dtype=torch.int32).reshape(n, 2))
        self.num_pairs = n
        return nat.step_layout(self.num_seqs, self.eng.num_q_heads, self.eng.num_kv_heads, self.eng.head_dim,
                               self.width, n)["bytes"]

    def h2d_bytes(self) -> int:
        """Bytes the staging kernel brings across the host link for the packed
        step: every field but the block tables whole, and of each table row
        the 16-byte words holding its entries up to ceil(context_len / 16)."""
        lay = nat.step_layout(self.num_seqs, self.eng.num_q_heads, self.eng.num_kv_heads, self.eng.head_dim,
                              self.width, self.num_pairs)
        dense = lay["bytes"] - (lay["context_lens"] - lay["block_tables"])
        ctx = self.field("context_lens").numpy().astype(np.int64)
        live = np.minimum(np.maximum((ctx + nat.BLOCK_TOKENS - 1) // nat.BLOCK_TOKENS, 0), self.width)
        start = lay["block_tables"] + np.arange(self.num_seqs, dtype=np.int64) * self.width * 4
        words = np.where(live > 0, (start + live * 4 + 15) // 16 - start // 16, 0)
        return int(dense + 16 * words.sum())

    def run(self, scale: float, num_ctas: int = 0, stream=None) -> torch.Tensor:
        """Enqueue the step; out_host holds the output once the stream passes it."""
        e = self.eng
        nat.decode_step_host(self.host, self.staging, self.num_pairs, e.k_cache, e.v_cache, self.width,
                             self.num_seqs, e.num_q_heads, scale, self.workspace, self.out_dev, self.out_host,
                             e.error, num_ctas, stream)
        return self.out_host
