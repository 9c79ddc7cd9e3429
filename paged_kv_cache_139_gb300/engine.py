"""A one-layer paged KV cache engine: the device K/V pools, the native block
allocator, and the decode step that ties the three device calls together.

One decode iteration ("vLLM & PagedAttention: Efficient Memory Management
for LLM Serving", §V): allocate physical blocks for the batch's new tokens
(copy-on-write where a sequence writes into a shared block, §VII), copy the
shared blocks, write the new keys and values at their slots, then run the
paged attention kernel over the block tables.  Host bookkeeping happens in
the native allocator; the four device steps run in libpkv's kernels.
"""
from __future__ import annotations

import dataclasses
import functools
from typing import Optional, Sequence

import numpy as np
import torch

import ctypes
import math

from . import (BlockAllocator, GrowingWorkspace, PkvError, _on, copy_blocks, kv_reshape_and_cache, kv_rotary_and_cache,
               kv_rotary_and_cache_fp8, kv_scales, make_fp8_workspace, make_workspace, paged_attention_decode,
               paged_attention_decode_fp8, paged_attention_decode_fp8_workspace_size, paged_attention_prefill,
               paged_attention_prefill_fp8, paged_attention_prefill_fp8_workspace_size, paged_attention_workspace_size,
               rotary_table, swap_blocks)
from ._lib import load


@dataclasses.dataclass
class RotaryPositions:
    """How a cache's queries and keys are rotated by their positions: the table
    of rotary_table and the layout of the pairs."""

    cos_sin: torch.Tensor     # float32 [positions][rotary_dim / 2][2]
    layout: str = "half"

    @classmethod
    def make(cls, num_positions: int, rotary_dim: int, device, layout: str = "half", **scaling) -> "RotaryPositions":
        """scaling: rotary_table's base, scaling, factor, ..."""
        return cls(rotary_table(num_positions, rotary_dim, device=device, **scaling), layout)


@dataclasses.dataclass
class StepPlan:
    """Host-side result of allocating one decode step."""

    seqs: np.ndarray          # int32 [n]
    slots: np.ndarray         # int64 [n]
    pairs: np.ndarray         # int32 [m][2] copy-on-write (src, dst)
    tables: np.ndarray        # int32 [n][max_blocks]
    context_lens: np.ndarray  # int32 [n]

    @property
    def positions(self) -> np.ndarray:
        """int32 [n]: the new tokens' positions."""
        return (self.context_lens - 1).astype(np.int32)


@dataclasses.dataclass
class DeviceStep:
    """The same plan on the device."""

    slots: torch.Tensor
    pairs: torch.Tensor
    tables: torch.Tensor
    context_lens: torch.Tensor
    max_context_len: int
    positions: Optional[torch.Tensor] = None     # int32, of a cache with rotary positions


@dataclasses.dataclass
class PrefillPlan:
    """Host-side result of allocating the new tokens of a prompt-phase step."""

    seqs: np.ndarray          # int32 [n]
    slots: np.ndarray         # int64 [T], sequence-major
    pairs: np.ndarray         # int32 [m][2] copy-on-write (src, dst)
    tables: np.ndarray        # int32 [n][max_blocks]
    context_lens: np.ndarray  # int32 [n]
    query_start: np.ndarray   # int32 [n + 1]

    @property
    def positions(self) -> np.ndarray:
        """int32 [T]: the new tokens' positions."""
        n = np.diff(self.query_start)
        return (np.arange(int(self.query_start[-1]))
                + np.repeat(self.context_lens - self.query_start[1:], n)).astype(np.int32)


@dataclasses.dataclass
class DevicePrefill:
    slots: torch.Tensor
    pairs: torch.Tensor
    tables: torch.Tensor
    context_lens: torch.Tensor
    query_start: torch.Tensor
    max_query_len: int
    max_context_len: int = 0
    positions: Optional[torch.Tensor] = None     # int32, of a cache with rotary positions


class StagedInputs:
    """A step's host inputs in one pinned buffer and their device copies in one
    device buffer, laid out alike (each tensor 256-byte aligned): a step then
    moves all its inputs with a single host-to-device copy instead of one per
    tensor.  Write the step's inputs into `host[name]`, call `upload()`, and
    pass `dev[name]` to the device calls."""

    def __init__(self, specs, device):
        """specs: {name: (shape, dtype)}."""
        self.device = torch.device(device)
        offs, off = {}, 0
        for name, (shape, dtype) in specs.items():
            n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
            offs[name] = (off, n, tuple(shape), dtype)
            off += (n + 255) // 256 * 256
        self.nbytes = off
        self._hbuf = torch.empty(max(off, 1), dtype=torch.uint8).pin_memory()
        self._dbuf = torch.empty(max(off, 1), dtype=torch.uint8, device=self.device)
        view = lambda buf, o, n, shape, dt: buf[o:o + n].view(dt).view(shape)
        self.host = {k: view(self._hbuf, *v) for k, v in offs.items()}
        self.dev = {k: view(self._dbuf, *v) for k, v in offs.items()}

    def upload(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        """One asynchronous copy of every input (on `stream`, default current)."""
        s = stream or torch.cuda.current_stream(self.device)
        with torch.cuda.stream(s):
            self._dbuf.copy_(self._hbuf, non_blocking=True)


class GraphStep:
    """A whole step -- one staged upload of its inputs, its device calls, the
    read-back of its output -- captured once in a CUDA graph and replayed:
    the GPU runs the copies and kernels back to back with no host round trip
    between them.  `prepare(stream)` must build the device calls (for example
    PagedKVCache.prepare / prepare_prefill) on the stream it is given, with
    the staged inputs' device views as arguments; the buffers must stay fixed
    (their contents may change between replays)."""

    def __init__(self, staged: StagedInputs, prepare, out: torch.Tensor, host_out: torch.Tensor, warmup: int = 2):
        dev = staged.device
        self._stream = torch.cuda.Stream(dev)
        self._prep = prepare(self._stream)
        self._staged, self._out, self._host_out = staged, out, host_out
        self._stream.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(self._stream):
            for _ in range(warmup):                  # first launches configure the kernels
                self._body()
        self._stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self._stream):
            self._body()
        self.device = dev

    def _body(self):
        self._staged.upload(self._stream)
        self._prep()
        self._host_out.copy_(self._out, non_blocking=True)

    def replay(self) -> None:
        self.graph.replay()


class HostKVPool:
    """The CPU side of swapping ("vLLM & PagedAttention" §VIII, Fig. 4): K and
    V pools in pinned host memory, which the GPU addresses directly, and the
    CPU block allocator that owns them."""

    def __init__(self, num_blocks: int, num_kv_heads: int, head_dim: int, block_size: int, dtype: torch.dtype,
                 free_order: Optional[Sequence[int]] = None):
        shape = (num_blocks, num_kv_heads, block_size, head_dim)
        self.key_cache = torch.empty(shape, dtype=dtype, pin_memory=True)
        self.value_cache = torch.empty(shape, dtype=dtype, pin_memory=True)
        # an 8-bit pool's block scales travel with the blocks
        self.scales = kv_scales(num_blocks, num_kv_heads, pin_memory=True) if dtype == torch.float8_e4m3fn else None
        self.alloc = BlockAllocator(num_blocks, block_size, free_order)
        self.num_blocks, self.block_size = num_blocks, block_size


class PagedKVCache:
    """dtype torch.float8_e4m3fn keeps keys and values in 8 bits with a scale
    per block and kv head (queries, keys and values come in 16 bits all the
    same).  With `rotary`, write, decode and prefill rotate queries and keys by
    their tokens' positions on the way.

    The 8-bit prompt phase's workspace holds the step's contexts in 16 bits.
    Caches whose calls follow one another on the GPU, as those of a model's
    layers do, need one between them: give the first layer's cache as
    `workspace_of` to the others."""

    def __init__(self, num_blocks: int, num_kv_heads: int, head_dim: int, block_size: int,
                 dtype: torch.dtype, device, max_blocks_per_seq: int,
                 free_order: Optional[Sequence[int]] = None,
                 key_cache: Optional[torch.Tensor] = None, value_cache: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, rotary: Optional[RotaryPositions] = None,
                 workspace_of: Optional["PagedKVCache"] = None):
        shape = (num_blocks, num_kv_heads, block_size, head_dim)
        self.device = torch.device(device)
        self.key_cache = key_cache if key_cache is not None else torch.empty(shape, dtype=dtype, device=self.device)
        self.value_cache = value_cache if value_cache is not None else torch.empty(shape, dtype=dtype,
                                                                                    device=self.device)
        assert tuple(self.key_cache.shape) == shape and tuple(self.value_cache.shape) == shape
        self.fp8 = dtype == torch.float8_e4m3fn
        self.scales = (scales if scales is not None else kv_scales(num_blocks, num_kv_heads, self.device)) if self.fp8 \
            else None
        if self.fp8:                     # prepared steps and block copies go by their address
            assert self.scales.shape == (num_blocks, num_kv_heads + num_kv_heads % 2, 2)
            assert self.scales.dtype == torch.float32 and self.key_cache.dtype == self.value_cache.dtype == dtype
            assert all(t.is_contiguous() for t in (self.scales, self.key_cache, self.value_cache))
        self.rotary = rotary
        self.alloc = BlockAllocator(num_blocks, block_size, free_order)
        self.num_blocks, self.num_kv_heads, self.head_dim, self.block_size = shape[0], shape[1], shape[3], shape[2]
        self.max_blocks_per_seq = max_blocks_per_seq
        self._ws: Optional[torch.Tensor] = None
        self._ws_retired: list = []
        self._swaps: list = []                        # (event after the copies, their pairs)
        self._ws8: Optional[GrowingWorkspace] = None
        if workspace_of is not None:
            if not (self.fp8 and workspace_of.fp8 and self.device == workspace_of.device):
                raise ValueError("workspace_of: 8-bit caches of one device share a workspace")
            self._ws8 = workspace_of._ws8
        elif self.fp8:
            self._ws8 = GrowingWorkspace(functools.partial(make_fp8_workspace, self.device))

    # -- host bookkeeping ------------------------------------------------------
    def new_sequence(self, length: int) -> int:
        return self.alloc.seq_new(length)

    def fork(self, seq: int) -> int:
        return self.alloc.fork(seq)

    def free(self, seq: int) -> None:
        self.alloc.free(seq)

    def plan_step(self, seqs: Sequence[int]) -> StepPlan:
        """Append one token to each sequence (all or nothing) and build the
        tables the attention kernel reads."""
        s = np.asarray(seqs, dtype=np.int32)
        slots, pairs = self.alloc.append_batch(s)
        tables, ctx = self.alloc.build_block_tables(s, self.max_blocks_per_seq)
        return StepPlan(s, slots, pairs, tables, ctx)

    def plan_beam_step(self, beams: Sequence[int], parents: Sequence[int]) -> StepPlan:
        """One beam-search step on the host: new candidate i continues
        beams[parents[i]] (fork where a parent has several children, prune
        the rest), each appends its token; the plan holds the new beams."""
        new, slots, pairs = self.alloc.beam_step(beams, parents)
        s = np.asarray(new, dtype=np.int32)
        tables, ctx = self.alloc.build_block_tables(s, self.max_blocks_per_seq)
        return StepPlan(s, slots, pairs, tables, ctx)

    def plan_tables(self, seqs: Sequence[int]) -> StepPlan:
        """Tables of the sequences as they stand (no new token)."""
        s = np.asarray(seqs, dtype=np.int32)
        tables, ctx = self.alloc.build_block_tables(s, self.max_blocks_per_seq)
        return StepPlan(s, np.empty(0, np.int64), np.empty((0, 2), np.int32), tables, ctx)

    def plan_prefill(self, seqs: Sequence[int], new_tokens: Sequence[int]) -> PrefillPlan:
        """Append new_tokens[i] tokens to seqs[i] (all or nothing): the prompt
        phase of a request, or its own input after a forked shared prefix."""
        s = np.asarray(seqs, dtype=np.int32)
        n = np.asarray(new_tokens, dtype=np.int64)
        slots, pairs = self.alloc.append_batch(np.repeat(s, n).astype(np.int32))
        tables, ctx = self.alloc.build_block_tables(s, self.max_blocks_per_seq)
        qs = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        return PrefillPlan(s, slots, pairs, tables, ctx, qs)

    def upload_prefill(self, plan: PrefillPlan, non_blocking: bool = False) -> DevicePrefill:
        d = self.device
        n = np.diff(plan.query_start)
        return DevicePrefill(
            slots=torch.from_numpy(plan.slots).to(d, non_blocking=non_blocking),
            pairs=torch.from_numpy(np.ascontiguousarray(plan.pairs)).to(d, non_blocking=non_blocking),
            tables=torch.from_numpy(plan.tables).to(d, non_blocking=non_blocking),
            context_lens=torch.from_numpy(plan.context_lens).to(d, non_blocking=non_blocking),
            query_start=torch.from_numpy(plan.query_start).to(d, non_blocking=non_blocking),
            max_query_len=int(n.max()) if n.size else 0,
            max_context_len=int(plan.context_lens.max()) if plan.context_lens.size else 0,
            positions=self._upload_positions(plan, non_blocking))

    def upload(self, plan: StepPlan, non_blocking: bool = False) -> DeviceStep:
        d = self.device
        return DeviceStep(
            slots=torch.from_numpy(plan.slots).to(d, non_blocking=non_blocking),
            pairs=torch.from_numpy(np.ascontiguousarray(plan.pairs)).to(d, non_blocking=non_blocking),
            tables=torch.from_numpy(plan.tables).to(d, non_blocking=non_blocking),
            context_lens=torch.from_numpy(plan.context_lens).to(d, non_blocking=non_blocking),
            max_context_len=int(plan.context_lens.max()) if plan.context_lens.size else 0,
            positions=self._upload_positions(plan, non_blocking) if plan.slots.size else None)

    def _upload_positions(self, plan, non_blocking: bool) -> Optional[torch.Tensor]:
        if self.rotary is None:
            return None
        return torch.from_numpy(plan.positions).to(self.device, non_blocking=non_blocking)

    # -- device steps ------------------------------------------------------------
    def workspace(self, num_seqs: int, num_heads: int, max_context_len: int, partition_size: int = 0):
        size = paged_attention_decode_fp8_workspace_size if self.fp8 else paged_attention_workspace_size
        return self._workspace(size(num_seqs, num_heads, self.num_kv_heads, self.head_dim, max_context_len,
                                    partition_size))

    def _workspace(self, need: int) -> torch.Tensor:
        if self.fp8:
            return self._ws8.get(need)
        if self._ws is None or self._ws.numel() < need:
            if self._ws is not None:
                self._ws_retired.append(self._ws)   # calls in flight on other streams may hold it
            self._ws = make_workspace(self.device, need)
        return self._ws

    def _pools(self):
        """What a block is made of: every pool that block copies and swaps move."""
        return (self.key_cache, self.value_cache) + ((self.scales,) if self.fp8 else ())

    def copy_on_write(self, pairs: torch.Tensor) -> None:
        if pairs.numel():
            for pool in self._pools():
                copy_blocks(pool, pairs)

    def write(self, key: torch.Tensor, value: torch.Tensor, slots: torch.Tensor,
              query: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
              query_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """The new tokens' keys and values into the cache.  Of a cache with
        rotary positions (which must be given), returns the rotated queries,
        in query_out if given; otherwise the queries as they are."""
        if self.rotary is None:
            if self.fp8:
                kv_rotary_and_cache_fp8(None, key, value, None, None, self.key_cache, self.value_cache, self.scales, slots)
            else:
                kv_reshape_and_cache(key, value, self.key_cache, self.value_cache, slots)
            return query
        r = self.rotary
        if self.fp8:
            return kv_rotary_and_cache_fp8(query, key, value, r.cos_sin, positions, self.key_cache, self.value_cache,
                                           self.scales, slots, layout=r.layout, query_out=query_out)
        return kv_rotary_and_cache(query, key, value, r.cos_sin, positions, self.key_cache, self.value_cache, slots,
                                   layout=r.layout, query_out=query_out)

    def attend(self, query: torch.Tensor, step: DeviceStep, out: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, partition_size: int = 0,
               max_context_len: Optional[int] = None) -> torch.Tensor:
        """Attention of queries as the cache's keys are: of a cache with
        rotary positions, rotated (as write returns them)."""
        if out is None:
            out = torch.empty_like(query)
        mcl = step.max_context_len if max_context_len is None else max_context_len
        mcl = mcl or _table_tokens(self, step)
        ws = self.workspace(query.shape[0], query.shape[1], mcl, partition_size)
        if self.fp8:
            return paged_attention_decode_fp8(out, query, self.key_cache, self.value_cache, self.scales, step.tables,
                                              step.context_lens, scale=scale, max_context_len=mcl,
                                              partition_size=partition_size, workspace=ws)
        return paged_attention_decode(out, query, self.key_cache, self.value_cache, step.tables,
                                      step.context_lens, scale=scale, max_context_len=mcl,
                                      partition_size=partition_size, workspace=ws)

    def decode(self, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, step: DeviceStep,
               out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
               partition_size: int = 0) -> torch.Tensor:
        """The device half of one decode iteration: copy-on-write copies, the
        new tokens' cache write, then attention (which reads the new tokens)."""
        self.copy_on_write(step.pairs)
        query = self.write(key, value, step.slots, query, step.positions)
        return self.attend(query, step, out, scale, partition_size)

    def prefill_workspace(self) -> torch.Tensor:
        """The prompt-phase attention's work counter (256 bytes, prepared
        once); the cache's prefill calls share it, one at a time."""
        if getattr(self, "_pf_ws", None) is None:
            self._pf_ws = make_workspace(self.device, 256)
        return self._pf_ws

    def prefill(self, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, step: DevicePrefill,
                out: Optional[torch.Tensor] = None, scale: Optional[float] = None) -> torch.Tensor:
        """The device half of a prompt-phase step: copy-on-write copies (a
        shared prefix's partly filled last block), the new tokens' cache write,
        then causal attention of the new tokens over the paged cache."""
        if out is None:
            out = torch.empty_like(query, memory_format=torch.contiguous_format)
        self.copy_on_write(step.pairs)
        query = self.write(key, value, step.slots, query, step.positions)
        if self.fp8:
            ws = self._workspace(paged_attention_prefill_fp8_workspace_size(
                step.context_lens.shape[0], self.num_kv_heads, self.head_dim, self.block_size,
                step.max_context_len or _table_tokens(self, step)))
            return paged_attention_prefill_fp8(out, query, self.key_cache, self.value_cache, self.scales, step.tables,
                                               step.context_lens, step.query_start, scale=scale,
                                               max_query_len=step.max_query_len, max_context_len=step.max_context_len,
                                               workspace=ws)
        return paged_attention_prefill(out, query, self.key_cache, self.value_cache, step.tables,
                                       step.context_lens, step.query_start, scale=scale,
                                       max_query_len=step.max_query_len, workspace=self.prefill_workspace())

    # -- swapping ----------------------------------------------------------------
    def _host_pools(self, host: HostKVPool):
        """The host pool's counterparts of _pools; before anything moves."""
        if self.fp8 != (host.scales is not None):
            raise ValueError("swapping between an 8-bit and a 16-bit pool")
        return (host.key_cache, host.value_cache) + ((host.scales,) if self.fp8 else ())

    def _keep_until_copied(self, pairs: torch.Tensor, stream) -> None:
        """The copies read the pairs from host memory, which would otherwise be
        given to the next swap's pairs while they run."""
        done = torch.cuda.Event()
        done.record(stream if stream is not None else torch.cuda.current_stream(self.device))
        self._swaps = [(e, p) for e, p in self._swaps if not e.query()] + [(done, pairs)]

    def swap_out(self, seqs: Sequence[int], host: HostKVPool, stream=None):
        """Evict a sequence group to the host pool, all or nothing: its blocks
        move to host blocks (one swap_blocks launch for keys, one for values)
        and the GPU blocks are freed.  Returns the group's ids in the host
        pool and the (GPU block, host block) pairs."""
        pools = self._host_pools(host)
        ids, pairs = self.alloc.move_group(host.alloc, seqs)
        if len(pairs):
            p = torch.from_numpy(pairs).pin_memory()
            for theirs, ours in zip(pools, self._pools()):
                swap_blocks(theirs, ours, p, stream)
            self._keep_until_copied(p, stream)
        return ids, pairs

    def swap_in(self, host_seqs: Sequence[int], host: HostKVPool, stream=None):
        """Bring a swapped-out group back: the reverse move and copies.
        Returns the group's GPU ids and the (host block, GPU block) pairs."""
        pools = self._host_pools(host)
        ids, pairs = host.alloc.move_group(self.alloc, host_seqs)
        if len(pairs):
            p = torch.from_numpy(pairs).pin_memory()
            for theirs, ours in zip(pools, self._pools()):
                swap_blocks(ours, theirs, p, stream)
            self._keep_until_copied(p, stream)
        return ids, pairs

    def prepare_prefill(self, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, step: DevicePrefill,
                        out: torch.Tensor, scale: Optional[float] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> "PreparedPrefill":
        """The device calls of a prompt-phase step on fixed buffers, with their
        C-ABI arguments built once."""
        return PreparedPrefill(self, query, key, value, step, out, scale, stream)

    def prepare(self, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, step: DeviceStep,
                out: torch.Tensor, scale: Optional[float] = None, partition_size: int = 0,
                stream: Optional[torch.cuda.Stream] = None, fused: bool = True) -> "PreparedStep":
        """The device calls of a decode step on fixed buffers, with their C-ABI
        arguments built once.  fused: the cache write rides in the attention
        launch (paged_attention_decode_write) when the step has one new token
        per sequence."""
        return PreparedStep(self, query, key, value, step, out, scale, partition_size, stream, fused)


def _table_tokens(eng: PagedKVCache, step) -> int:
    """What bounds a step's contexts when nothing else does (a bound of 0, as of
    sequences without tokens, is none to the calls); it sizes the workspace."""
    return step.tables.shape[1] * eng.block_size


def _check_step(eng: PagedKVCache, query, key, value, step, out, extra=()) -> int:
    """The dtype code of a prepared step's 16-bit tensors, which must be on the GPU and contiguous."""
    d = query.shape[2]
    assert out.shape == query.shape and out.dtype == query.dtype == key.dtype == value.dtype
    assert eng.fp8 or query.dtype == eng.key_cache.dtype
    assert query.dtype in (torch.float16, torch.bfloat16)
    assert key.shape == value.shape == (step.slots.shape[0], eng.num_kv_heads, d)
    for t in (query, key, value, out, step.slots, step.tables, step.context_lens, step.pairs, *extra):
        assert t.is_cuda and t.is_contiguous()
    if eng.rotary is not None:
        assert query.shape[0] == key.shape[0], "rotary positions: a query for each new token"
        pos, cs = step.positions, eng.rotary.cos_sin
        assert pos is not None and pos.shape == step.slots.shape
        assert cs.dim() == 3 and cs.shape[2] == 2 and eng.rotary.layout in ("half", "interleaved")
        for t, dtype in ((pos, torch.int32), (cs, torch.float32)):
            assert t.dtype == dtype and t.device == query.device and t.is_contiguous()
    return 1 if query.dtype == torch.bfloat16 else 0


def _held(eng: PagedKVCache, ws, stream):
    """The cache's own tensors whose addresses a prepared step holds: it keeps
    them, since the cache may be given others (a longer table, a larger
    workspace) or go.  Made on other streams than the step's, their memory is
    not used again before the step's work is done, if the step is dropped
    while that runs."""
    held = (ws, *eng._pools(), *((eng.rotary.cos_sin,) if eng.rotary else ()))
    for t in held:
        t.record_stream(stream)
    return held


def _scratch_queries(eng: PagedKVCache, query, stream):
    """The queries as a prepared step's attention reads them: with rotary
    positions a tensor of the step's own, made on its stream."""
    if eng.rotary is None:
        return query
    with _on(stream):
        return torch.empty_like(query)


def _copy_calls(eng: PagedKVCache, step, st):
    n = step.pairs.shape[0] if step.pairs.dim() == 2 else 0
    return [(c.data_ptr(), step.pairs.data_ptr(), n, c.numel() // c.shape[0] * c.element_size(), eng.num_blocks, st)
            for c in eng._pools()] if n else []


def _write_call(eng: PagedKVCache, query, query_out, key, value, step, code, st):
    """The C call of PagedKVCache.write and its arguments."""
    T, Hkv, d, B, NB = step.slots.shape[0], eng.num_kv_heads, eng.head_dim, eng.block_size, eng.num_blocks
    ptrs = (key.data_ptr(), value.data_ptr(), eng.key_cache.data_ptr(), eng.value_cache.data_ptr())
    if eng.rotary is None and not eng.fp8:
        return "kv_reshape_and_cache", (*ptrs, step.slots.data_ptr(), T, Hkv, d, B, NB, code, st)
    r = eng.rotary
    H, rot, npos = (query.shape[1], 2 * r.cos_sin.shape[1], r.cos_sin.shape[0]) if r else (0, 0, 0)
    args = (query_out.data_ptr() if r else None, query.data_ptr() if r else None, *ptrs,
            *((eng.scales.data_ptr(),) if eng.fp8 else ()), r.cos_sin.data_ptr() if r else None,
            step.positions.data_ptr() if r else None, step.slots.data_ptr(), T, H, Hkv, d, rot, npos,
            ("half", "interleaved").index(r.layout) if r else 0, H * d, Hkv * d, Hkv * d, B, NB, code, st)
    return ("kv_rotary_and_cache_fp8" if eng.fp8 else "kv_rotary_and_cache"), args


class PreparedStep:
    """copy_blocks, the cache write and the attention for one set of buffers,
    their arguments checked and marshalled once: issuing the step then costs
    three or four plain C calls.  For decode loops that run the same buffers
    every iteration (the buffers' contents may change).  The step holds its
    rotated queries and its workspace: a CUDA graph that has captured its
    calls is replayed only while it lives."""

    def __init__(self, eng: PagedKVCache, query, key, value, step: DeviceStep, out, scale, partition_size, stream,
                 fused=True):
        self._L = load()
        S, H, d = query.shape
        code = _check_step(eng, query, key, value, step, out)
        stream = stream if stream is not None else torch.cuda.current_stream(eng.device)
        st = ctypes.c_void_p(stream.cuda_stream)
        mcl = step.max_context_len or _table_tokens(eng, step)
        ws = eng.workspace(S, H, mcl, partition_size)
        q = _scratch_queries(eng, query, stream)
        self._keep = (query, q, key, value, step, out, _held(eng, ws, stream))
        NB, B = eng.num_blocks, eng.block_size
        self._copy = _copy_calls(eng, step, st)
        T = self._tokens = step.slots.shape[0]
        self._write_name, self._write = _write_call(eng, query, q, key, value, step, code, st)
        self._attend_name = "paged_attention_decode_fp8" if eng.fp8 else "paged_attention_decode"
        self._attend = (out.data_ptr(), q.data_ptr(), eng.key_cache.data_ptr(), eng.value_cache.data_ptr(),
                        *((eng.scales.data_ptr(),) if eng.fp8 else ()),
                        step.tables.data_ptr(), step.context_lens.data_ptr(), S, step.tables.shape[1],
                        mcl, B, NB, H, eng.num_kv_heads, d,
                        float(1.0 / math.sqrt(d) if scale is None else scale), partition_size, ws.data_ptr(),
                        ws.numel(), code, st)
        # one new token per sequence, in sequence order, written as it is in 16 bits: the write can ride in the
        # attention launch
        self._write_attend = None
        if T == S and not eng.fp8 and eng.rotary is None:
            self._write_attend = (out.data_ptr(), query.data_ptr(), key.data_ptr(), value.data_ptr(),
                                  eng.key_cache.data_ptr(), eng.value_cache.data_ptr(), step.slots.data_ptr(),
                                  step.tables.data_ptr(), step.context_lens.data_ptr(), S, step.tables.shape[1],
                                  mcl, B, NB, H, eng.num_kv_heads, d,
                                  float(1.0 / math.sqrt(d) if scale is None else scale), partition_size, ws.data_ptr(),
                                  ws.numel(), code, st)
        self._fused = fused and self._write_attend is not None

    def copy(self) -> None:
        for args in self._copy:
            rc = self._L.copy_blocks(*args)
            if rc:
                raise PkvError(rc, "copy_blocks")

    def write(self) -> None:
        if self._tokens:
            rc = getattr(self._L, self._write_name)(*self._write)
            if rc:
                raise PkvError(rc, self._write_name)

    def attend(self) -> None:
        rc = getattr(self._L, self._attend_name)(*self._attend)
        if rc:
            raise PkvError(rc, self._attend_name)

    def write_attend(self) -> None:
        """The cache write and the attention in one launch (paged_attention_decode_write): of a 16-bit cache without
        rotary positions, for a step of one token per sequence."""
        if self._write_attend is None:
            raise ValueError("write_attend: only a 16-bit cache without rotary positions, one new token per sequence, is "
                             "written in the attention launch")
        rc = self._L.paged_attention_decode_write(*self._write_attend)
        if rc:
            raise PkvError(rc, "paged_attention_decode_write")

    def front(self) -> None:
        """What runs before the attention launch: the copies (and the write when not fused)."""
        self.copy()
        if not self._fused:
            self.write()

    def back(self) -> None:
        """The attention launch (with the write when fused)."""
        if self._fused:
            self.write_attend()
        else:
            self.attend()

    def __call__(self) -> None:
        self.front()
        self.back()


class PreparedPrefill:
    """copy_blocks, the cache write and the prompt-phase attention for one set
    of buffers, their arguments checked and marshalled once."""

    def __init__(self, eng: PagedKVCache, query, key, value, step: DevicePrefill, out, scale, stream):
        self._L = load()
        T, H, d = query.shape
        code = _check_step(eng, query, key, value, step, out, (step.query_start,))
        stream = stream if stream is not None else torch.cuda.current_stream(eng.device)
        st = ctypes.c_void_p(stream.cuda_stream)
        S = step.context_lens.shape[0]
        NB, B, mb = eng.num_blocks, eng.block_size, step.tables.shape[1]
        if eng.fp8:
            ws = eng._workspace(paged_attention_prefill_fp8_workspace_size(
                S, eng.num_kv_heads, d, B, step.max_context_len or _table_tokens(eng, step)))
        else:
            ws = eng.prefill_workspace()
        q = _scratch_queries(eng, query, stream)
        self._keep = (query, q, key, value, step, out, _held(eng, ws, stream))
        self._copy = _copy_calls(eng, step, st)
        self._tokens = step.slots.shape[0]
        self._write_name, self._write = _write_call(eng, query, q, key, value, step, code, st)
        self._attend_name = "paged_attention_prefill_fp8" if eng.fp8 else "paged_attention_prefill"
        self._attend = (out.data_ptr(), q.data_ptr(), eng.key_cache.data_ptr(), eng.value_cache.data_ptr(),
                        *((eng.scales.data_ptr(),) if eng.fp8 else ()),
                        step.tables.data_ptr(), step.context_lens.data_ptr(), step.query_start.data_ptr(), S, T,
                        step.max_query_len, *((step.max_context_len,) if eng.fp8 else ()), mb, B, NB, H,
                        eng.num_kv_heads, d, float(1.0 / math.sqrt(d) if scale is None else scale), ws.data_ptr(),
                        ws.numel(), code, st)

    copy, write, attend = PreparedStep.copy, PreparedStep.write, PreparedStep.attend

    def __call__(self) -> None:
        self.copy()
        self.write()
        self.attend()
