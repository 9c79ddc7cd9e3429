"""paged_kv_cache_139_gb300 -- the decode hot path of PagedAttention on GB300.

A thin Python binding of libpkv.so (declared in include/pkv.h).  Every
function here only checks and marshals its arguments -- torch tensors to
device pointers, the current CUDA stream -- and calls the C entry point of
the same name; all the work runs in the library's sm_103a kernels.  PyTorch
provides device memory and streams.  There is no fallback: if the library is
missing, the first call raises.

    kv_reshape_and_cache     slot-mapped K/V write into the paged cache
    paged_attention_decode   block-table gather + decode attention
    copy_blocks              copy-on-write block copy
    BlockAllocator           the native ref-counted block allocator
    rotary_table             cosines and sines of the rotary positions
    kv_rotary_and_cache      the K/V write with the rotary rotation on the way
    *_fp8                    the K/V write and the attention of an 8-bit cache
    *_window                 decode and prompt-phase attention with a sliding window and sinks
    paged_attention_decode_shared   decode attention that reads shared prefixes once
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import re
import threading
import weakref
from typing import Optional, Sequence

import numpy as np
import torch

from ._lib import STATUS, load

__all__ = ["PkvError", "PkvOOM", "kv_reshape_and_cache", "paged_attention_decode",
           "paged_attention_decode_noalloc", "paged_attention_decode_write", "paged_attention_prefill", "paged_attention_workspace_size",
           "make_workspace",
           "paged_attention_partition_size", "copy_blocks",
           "rotary_table", "kv_rotary_and_cache", "kv_rotary_and_cache_fp8", "kv_scales",
           "paged_attention_decode_fp8", "paged_attention_decode_fp8_workspace_size",
           "paged_attention_prefill_fp8", "paged_attention_prefill_fp8_workspace_size", "make_fp8_workspace", "GrowingWorkspace",
           "paged_attention_decode_window", "paged_attention_prefill_window", "paged_attention_decode_shared",
           "paged_attention_decode_shared_workspace_size",
           "validate_copy_pairs", "swap_blocks", "check", "launch_count", "version", "BlockAllocator", "library_path"]

PKV_F16, PKV_BF16 = 0, 1


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        self.status_name = STATUS.get(status, str(status))
        super().__init__(f"{what}: {self.status_name}: {load().pkv_last_error_string().decode()}")


class PkvOOM(PkvError):
    """The allocator has too few free blocks; its state is unchanged."""


def _ck(rc: int, what: str) -> None:
    if rc != 0:
        raise (PkvOOM if rc == 2 else PkvError)(rc, what)


def library_path() -> str:
    from ._lib import LIB_PATH
    return str(LIB_PATH)


def version() -> int:
    return load().pkv_version()


def launch_count() -> int:
    """Kernels launched by the library in this process."""
    return int(load().pkv_launch_count())


# -- marshalling -----------------------------------------------------------------

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return PKV_F16
    if t.dtype == torch.bfloat16:
        return PKV_BF16
    raise TypeError(f"expected float16 or bfloat16, got {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None, ndim=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    return t.data_ptr()


def _stream(stream: Optional[torch.cuda.Stream], device) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream: Optional[torch.cuda.Stream]):
    """Where memory is made for a call on `stream`: taken from the current
    stream's, work still queued there could be using it while the call writes."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


# -- the three device calls -------------------------------------------------------

def kv_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                         value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """key/value [T][Hkv][d]; caches [NB][Hkv][B][d]; slot_mapping int64 [T]."""
    NB, Hkv, B, d = key_cache.shape
    T = key.shape[0]
    if tuple(key.shape) != (T, Hkv, d) or key.shape != value.shape or value_cache.shape != key_cache.shape:
        raise ValueError("kv_reshape_and_cache: shape mismatch")
    if key.dtype != key_cache.dtype or value.dtype != key_cache.dtype or value_cache.dtype != key_cache.dtype:
        raise TypeError("kv_reshape_and_cache: dtype mismatch")
    if slot_mapping.shape != (T,):
        raise ValueError("kv_reshape_and_cache: slot_mapping must be [num_tokens]")
    args = (_dev(key, "key"), _dev(value, "value"), _dev(key_cache, "key_cache"),
            _dev(value_cache, "value_cache"), _dev(slot_mapping, "slot_mapping", torch.int64))
    rc = load().kv_reshape_and_cache(*args, T, Hkv, d, B, NB, _dtype_code(key_cache),
                                     _stream(stream, key_cache.device))
    _ck(rc, "kv_reshape_and_cache")


def paged_attention_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                   max_context_len: int, partition_size: int = 0) -> int:
    return int(load().paged_attention_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                     max_context_len, partition_size))


def paged_attention_partition_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                   max_context_len: int, partition_size: int = 0) -> int:
    return int(load().paged_attention_partition_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                     max_context_len, partition_size))


def make_workspace(device, nbytes: int, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """A device buffer of at least nbytes, prepared for paged_attention_decode
    and paged_attention_prefill (paged_attention_workspace_init).  Returns
    once the preparation has finished, so any stream may use the buffer."""
    dev = torch.device(device)
    with _on(stream):
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    st = _stream(stream, dev)
    _ck(load().paged_attention_workspace_init(buf.data_ptr(), buf.numel(), st), "paged_attention_workspace_init")
    (stream or torch.cuda.current_stream(dev)).synchronize()
    return _made(buf, "paged_attention_workspace_init")


_workspaces: list = []


def _made(buf: torch.Tensor, init: str) -> torch.Tensor:
    """Remembers a workspace, for as long as it lives, and the call that prepares it."""
    _workspaces[:] = [(ref, name) for ref, name in _workspaces if ref() is not None]
    _workspaces.append((weakref.ref(buf), init))
    return buf


def _prepare_again(index: int) -> None:
    """Every workspace made here for this device: a call that gave up waiting
    leaves the counters of its own mid-count, and later calls on it would skip
    work."""
    torch.cuda.synchronize(index)
    for ref, init in _workspaces:
        buf = ref()
        if buf is not None and buf.get_device() == index:
            _call(getattr(load(), init), init, index, buf.data_ptr(), buf.numel(), _raw_stream(None, index))
    torch.cuda.synchronize(index)


_ws_cache: dict = {}
_ws_retired: list = []


def _workspace(device, nbytes: int) -> torch.Tensor:
    """The binding's own workspace: at least nbytes, kept per device.  A
    buffer replaced by a larger one is kept alive, since calls on other
    streams may still be using it (the sizes only grow, so few are kept)."""
    key = torch.device(device)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        if buf is not None:
            _ws_retired.append(buf)
        buf = make_workspace(key, nbytes)
        _ws_cache[key] = buf
    return buf


def paged_attention_decode(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                           value_cache: torch.Tensor, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, scale: Optional[float] = None,
                           max_context_len: int = 0, partition_size: int = 0,
                           workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out/query [S][H][d]; caches [NB][Hkv][B][d]; block_tables int32 [S][MB];
    context_lens int32 [S].  scale defaults to 1/sqrt(d).  A workspace passed
    in must come from make_workspace (or paged_attention_workspace_init) and
    serve one call at a time; None takes the binding's own per-device buffer,
    which every decode and prefill call without a workspace shares, so calls
    through it must not overlap on the GPU (give calls on concurrent streams
    a workspace each).  Returns out."""
    S, H, d = query.shape
    NB, Hkv, B, d2 = key_cache.shape
    if d2 != d or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise ValueError("paged_attention_decode: shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("paged_attention_decode: block_tables must be [S][max_blocks], context_lens [S]")
    if not (query.dtype == out.dtype == key_cache.dtype == value_cache.dtype):
        raise TypeError("paged_attention_decode: dtype mismatch")
    mb = block_tables.shape[1]
    mcl = max_context_len if max_context_len > 0 else mb * B
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = _workspace(query.device, paged_attention_workspace_size(S, H, Hkv, d, mcl, partition_size))
    ws_ptr = _dev(workspace, "workspace")
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().paged_attention_decode(
        _dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"),
        _dev(block_tables, "block_tables", torch.int32), _dev(context_lens, "context_lens", torch.int32),
        S, mb, max_context_len, B, NB, H, Hkv, d, float(scale), partition_size, ws_ptr, ws_bytes,
        _dtype_code(query), _stream(stream, query.device))
    _ck(rc, "paged_attention_decode")
    return out


def paged_attention_decode_write(out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                                 key_cache: torch.Tensor, value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                                 block_tables: torch.Tensor, context_lens: torch.Tensor,
                                 scale: Optional[float] = None, max_context_len: int = 0, partition_size: int = 0,
                                 workspace: Optional[torch.Tensor] = None,
                                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """kv_reshape_and_cache of each sequence's new token (key/value [S][Hkv][d],
    slot_mapping int64 [S], the slot of position context_lens[s] - 1) and
    paged_attention_decode in one launch.  workspace as for
    paged_attention_decode: None shares the binding's per-device buffer, so
    calls through it must not overlap on the GPU.  Returns out."""
    S, H, d = query.shape
    NB, Hkv, B, d2 = key_cache.shape
    if d2 != d or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise ValueError("paged_attention_decode_write: shape mismatch")
    if key.shape != (S, Hkv, d) or value.shape != key.shape or slot_mapping.shape != (S,):
        raise ValueError("paged_attention_decode_write: key/value must be [S][Hkv][d], slot_mapping [S]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("paged_attention_decode_write: block_tables must be [S][max_blocks], context_lens [S]")
    mb = block_tables.shape[1]
    mcl = max_context_len if max_context_len > 0 else mb * B
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = _workspace(query.device, paged_attention_workspace_size(S, H, Hkv, d, mcl, partition_size))
    rc = load().paged_attention_decode_write(
        _dev(out, "out"), _dev(query, "query"), _dev(key, "key"), _dev(value, "value"),
        _dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"),
        _dev(slot_mapping, "slot_mapping", torch.int64), _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32), S, mb, max_context_len, B, NB, H, Hkv, d, float(scale),
        partition_size, _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _dtype_code(query), _stream(stream, query.device))
    _ck(rc, "paged_attention_decode_write")
    return out


def paged_attention_prefill(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                            value_cache: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, query_start: torch.Tensor,
                            scale: Optional[float] = None, max_query_len: int = 0,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Prompt-phase attention: out/query [T][H][d] hold the new tokens of all
    sequences back to back, query_start int32 [S+1] their offsets; the new
    tokens of sequence s are the last n_s of its context_lens[s] and each
    attends every token up to its own position.  Their keys and values must
    already be in the cache.  workspace: a buffer from make_workspace (its
    counter balances the work over the SMs), serving one call at a time; None
    takes the binding's own per-device buffer, which paged_attention_decode
    calls share (calls through it must not overlap on the GPU).  Returns out."""
    T, H, d = query.shape
    NB, Hkv, B, d2 = key_cache.shape
    S = context_lens.shape[0]
    if d2 != d or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise ValueError("paged_attention_prefill: shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or query_start.shape != (S + 1,):
        raise ValueError("paged_attention_prefill: block_tables must be [S][max_blocks], query_start [S+1]")
    if not (query.dtype == out.dtype == key_cache.dtype == value_cache.dtype):
        raise TypeError("paged_attention_prefill: dtype mismatch")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    ws = _workspace(query.device, 256) if workspace is None else workspace
    rc = load().paged_attention_prefill(
        _dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"),
        _dev(block_tables, "block_tables", torch.int32), _dev(context_lens, "context_lens", torch.int32),
        _dev(query_start, "query_start", torch.int32), S, T, max_query_len, block_tables.shape[1], B, NB, H, Hkv,
        d, float(scale), _dev(ws, "workspace", torch.uint8), ws.numel(), _dtype_code(query),
        _stream(stream, query.device))
    _ck(rc, "paged_attention_prefill")
    return out


def paged_attention_decode_noalloc(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, block_tables: torch.Tensor,
                                   context_lens: torch.Tensor, scale: Optional[float] = None,
                                   max_context_len: int = 0, partition_size: int = 0,
                                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """paged_attention_decode without a workspace: for callers that may not
    allocate device memory when they run attention.  The partition partials
    use the library's built-in 16 MiB device array, shared by every call on a
    device (one call at a time); larger sizes raise PkvError (PKV_EINVAL).
    The first call on a device, and the first after check() reported a
    device-wait timeout, prepares the array and waits for it, so it must not
    run during stream capture (PkvError, PKV_EINVAL)."""
    S, H, d = query.shape
    NB, Hkv, B, d2 = key_cache.shape
    if d2 != d or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise ValueError("paged_attention_decode_noalloc: shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("paged_attention_decode_noalloc: block_tables must be [S][max_blocks], context_lens [S]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rc = load().paged_attention_decode_noalloc(
        _dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"),
        _dev(block_tables, "block_tables", torch.int32), _dev(context_lens, "context_lens", torch.int32),
        S, block_tables.shape[1], max_context_len, B, NB, H, Hkv, d, float(scale), partition_size,
        _dtype_code(query), _stream(stream, query.device))
    _ck(rc, "paged_attention_decode_noalloc")
    return out


# -- rotary positions ---------------------------------------------------------------

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "by_parts": 2}


def _raw_stream(stream: Optional[torch.cuda.Stream], index: int) -> int:
    """The stream's handle; the current one's without building a Stream."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)


def _call(fn, what: str, index: int, *args) -> None:
    """A C call on the tensors' own device: the library launches on the current one."""
    was = torch.cuda.current_device()
    if was == index:
        rc = fn(*args)
    else:
        torch.cuda.set_device(index)
        try:
            rc = fn(*args)
        finally:
            torch.cuda.set_device(was)
    if rc:
        _ck(rc, what)


def _at(t: torch.Tensor, name: str, dtype, index: int) -> int:
    """The address of a contiguous tensor of this type on CUDA device `index`."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.is_contiguous():
        return t.data_ptr()
    ptr = _dev(t, name, dtype)                      # says what is wrong
    raise ValueError(f"{name} (at {ptr:#x}) is on {t.device}, other tensors on cuda:{index}")


def _rows(t: torch.Tensor, name: str, dtype, index: int, T: int, h: int, d: int):
    """Pointer and token stride of a [T][h][d] tensor whose tokens may lie
    further apart than h * d elements (a slice of a wider projection)."""
    if t.shape != (T, h, d):
        raise ValueError(f"{name} must be [{T}][{h}][{d}], got shape {tuple(t.shape)}")
    if t.dtype is not dtype or t.get_device() != index:
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{index}")
    st, sh, sd = t.stride()
    if T <= 1:
        st = h * d
    if T and ((h > 1 and sh != d) or sd != 1 or st < h * d or st % 8):
        raise ValueError(f"{name}: a token's heads must be contiguous, tokens a multiple of 8 elements apart")
    return t.data_ptr(), st


def _cuda_index(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def rotary_table(num_positions: int, rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, original_positions: int = 0, low_turns: float = 1.0, high_turns: float = 32.0,
                 magnitude: float = 1.0, device="cuda", out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """fp32 [num_positions][rotary_dim / 2][2]: magnitude * (cos, sin) of
    position times theta_i, theta_i = base^(-2i / rotary_dim), scaled for long
    contexts: "none", "linear" (theta / factor), or "by_parts" (pairs that turn
    at least high_turns times over original_positions keep their angle, those
    below low_turns are divided by factor, a ramp between).  Written into out
    when given, else into a tensor allocated on the call's stream."""
    if scaling not in _SCALINGS:
        raise ValueError(f"rotary_table: scaling {scaling!r} not one of {sorted(_SCALINGS)}")
    if out is None:
        with _on(stream):
            out = torch.empty(num_positions, rotary_dim // 2, 2, dtype=torch.float32, device=device)
    elif out.shape != (num_positions, rotary_dim // 2, 2):
        raise ValueError("rotary_table: out must be [num_positions][rotary_dim / 2][2]")
    index = _cuda_index(out, "out")
    _call(load().rotary_table, "rotary_table", index, _at(out, "out", torch.float32, index), num_positions, rotary_dim,
          base, _SCALINGS[scaling], factor, original_positions, low_turns, high_turns, magnitude,
          _raw_stream(stream, index))
    return out


def kv_scales(num_blocks: int, num_kv_heads: int, device="cuda", pin_memory: bool = False) -> torch.Tensor:
    """The block scales of an 8-bit cache, zero: fp32
    [num_blocks][num_kv_heads rounded up to even][2] (key, value)."""
    return torch.zeros(num_blocks, num_kv_heads + num_kv_heads % 2, 2, dtype=torch.float32,
                       device="cpu" if pin_memory else device, pin_memory=pin_memory)


def _append(what, fp8, query, key, value, cos_sin, positions, key_cache, value_cache, scales, slot_mapping, layout,
            query_out, stream):
    if layout not in _LAYOUTS:
        raise ValueError(f"{what}: layout {layout!r} not one of {sorted(_LAYOUTS)}")
    index = _cuda_index(key_cache, "key_cache")
    NB, Hkv, B, d = key_cache.shape
    T, dtype = key.shape[0], key.dtype
    if value_cache.shape != key_cache.shape or slot_mapping.shape != (T,):
        raise ValueError(f"{what}: caches of different shapes, or slot_mapping not [num_tokens]")
    code = _dtype_code(key)
    k_ptr, k_stride = _rows(key, "key", dtype, index, T, Hkv, d)
    v_ptr, v_stride = _rows(value, "value", dtype, index, T, Hkv, d)
    rot = npos = H = q_stride = 0
    cs_ptr = pos_ptr = q_ptr = qo_ptr = None
    if cos_sin is not None:
        if cos_sin.dim() != 3 or cos_sin.shape[2] != 2 or positions is None or positions.shape != (T,):
            raise ValueError(f"{what}: cos_sin must be [positions][rotary_dim / 2][2], positions [num_tokens]")
        npos, rot = cos_sin.shape[0], 2 * cos_sin.shape[1]
        cs_ptr = _at(cos_sin, "cos_sin", torch.float32, index)
        pos_ptr = _at(positions, "positions", torch.int32, index)
    if query is not None:
        if cos_sin is None:
            raise ValueError(f"{what}: a query needs a table to rotate it by")
        H = query.shape[1]
        q_ptr, q_stride = _rows(query, "query", dtype, index, T, H, d)
        if query_out is None:
            with _on(stream):
                query_out = torch.empty(T, H, d, dtype=dtype, device=key_cache.device)
        elif query_out.shape != query.shape:
            raise ValueError(f"{what}: query_out must be shaped like query")
        qo_ptr = _at(query_out, "query_out", dtype, index)
    cache_dtype = torch.float8_e4m3fn if fp8 else dtype
    caches = _at(key_cache, "key_cache", cache_dtype, index), _at(value_cache, "value_cache", cache_dtype, index)
    slots = _at(slot_mapping, "slot_mapping", torch.int64, index)
    L = load()
    if fp8:
        if scales.shape != (NB, Hkv + Hkv % 2, 2):
            raise ValueError(f"{what}: scales must be [num_blocks][num_kv_heads rounded up to even][2]")
        _call(L.kv_rotary_and_cache_fp8, what, index, qo_ptr, q_ptr, k_ptr, v_ptr, *caches,
              _at(scales, "scales", torch.float32, index), cs_ptr, pos_ptr, slots, T, H, Hkv, d, rot, npos,
              _LAYOUTS[layout], q_stride, k_stride, v_stride, B, NB, code, _raw_stream(stream, index))
    else:
        _call(L.kv_rotary_and_cache, what, index, qo_ptr, q_ptr, k_ptr, v_ptr, *caches, cs_ptr, pos_ptr, slots, T, H,
              Hkv, d, rot, npos, _LAYOUTS[layout], q_stride, k_stride, v_stride, B, NB, code,
              _raw_stream(stream, index))
    return query_out


def kv_rotary_and_cache(query: Optional[torch.Tensor], key: torch.Tensor, value: torch.Tensor, cos_sin: torch.Tensor,
                        positions: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                        slot_mapping: torch.Tensor, layout: str = "half", query_out: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """Rotate query [T][H][d] (None: keys only) and key [T][Hkv][d] by their
    tokens' positions (int32 [T]) and write the keys and values at their slots,
    in one launch.  cos_sin comes from rotary_table; layout "half" pairs (i,
    i + rotary_dim / 2), "interleaved" (2i, 2i + 1).  query, key and value may
    be slices of one projection's rows.  Returns the rotated queries
    (query_out, which may be a contiguous query itself; without it, a tensor
    allocated on the call's stream)."""
    if cos_sin is None:
        raise ValueError("kv_rotary_and_cache: needs a table (kv_reshape_and_cache writes without rotation)")
    return _append("kv_rotary_and_cache", False, query, key, value, cos_sin, positions, key_cache, value_cache, None,
                   slot_mapping, layout, query_out, stream)


def kv_rotary_and_cache_fp8(query: Optional[torch.Tensor], key: torch.Tensor, value: torch.Tensor,
                            cos_sin: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                            key_cache: torch.Tensor, value_cache: torch.Tensor, scales: torch.Tensor,
                            slot_mapping: torch.Tensor, layout: str = "half",
                            query_out: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """kv_rotary_and_cache into an 8-bit cache: float8_e4m3fn caches
    [NB][Hkv][B][d] and their block scales (kv_scales), which the call keeps.
    cos_sin, positions and query None: append without rotation.  The tokens of
    one block must stand next to one another in slot_mapping."""
    return _append("kv_rotary_and_cache_fp8", True, query, key, value, cos_sin, positions, key_cache, value_cache,
                   scales, slot_mapping, layout, query_out, stream)


# -- attention over an 8-bit cache ---------------------------------------------------

@functools.lru_cache(maxsize=4096)
def paged_attention_decode_fp8_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                              max_context_len: int, partition_size: int = 0) -> int:
    return int(load().paged_attention_decode_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                                max_context_len, partition_size))


@functools.lru_cache(maxsize=4096)
def paged_attention_prefill_fp8_workspace_size(num_seqs: int, num_kv_heads: int, head_dim: int, block_size: int,
                                               max_context_len: int) -> int:
    return int(load().paged_attention_prefill_fp8_workspace_size(num_seqs, num_kv_heads, head_dim, block_size,
                                                                 max_context_len))


def make_fp8_workspace(device, nbytes: int, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """A device buffer of at least nbytes, prepared for
    paged_attention_decode_fp8 and paged_attention_prefill_fp8.  Returns once
    the preparation has finished, so any stream may use the buffer."""
    with _on(stream):
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=torch.device(device))
    index = buf.get_device()
    _call(load().paged_attention_fp8_workspace_init, "paged_attention_fp8_workspace_init", index, buf.data_ptr(),
          buf.numel(), _raw_stream(stream, index))
    (stream or torch.cuda.current_stream(buf.device)).synchronize()
    return _made(buf, "paged_attention_fp8_workspace_init")


def _capturing(stream: Optional[torch.cuda.Stream]) -> bool:
    """Whether the call's stream (or the current one, which the call may be forked from) is being captured."""
    if torch.cuda.is_current_stream_capturing():
        return True
    if stream is None:
        return False
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class GrowingWorkspace:
    """One workspace for 8-bit calls that follow one another, made by
    make(nbytes) and grown as they need.  The prompt phase keeps whole contexts
    in it, and a prompt in chunks asks for a little more each time: it grows by
    half at least, and the smaller one is let go when the device has done all
    that may still use it.  One that a CUDA graph has captured is kept, since
    the graph holds its address."""

    def __init__(self, make):
        self._make = make
        self._buf: Optional[torch.Tensor] = None
        self._captured = False
        self._kept: list = []

    def get(self, nbytes: int, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """At least nbytes, for a call on `stream` (default the current one)."""
        capturing = _capturing(stream)
        if self._buf is None or self._buf.numel() < nbytes:
            if capturing:
                raise RuntimeError(f"a workspace of {nbytes} bytes cannot be made during a stream capture: make the call "
                                   "once before, or give it a workspace")
            self._grow(nbytes)
        self._captured |= capturing
        return self._buf

    def _grow(self, nbytes: int) -> None:
        want = nbytes
        if self._buf is not None:
            want = max(nbytes, self._buf.numel() * 3 // 2)
            if self._captured:
                self._kept.append(self._buf)
            else:
                torch.cuda.synchronize(self._buf.device)
            self._buf, self._captured = None, False           # before the larger one is made
        try:
            self._buf = self._make(want)
        except torch.OutOfMemoryError:
            if want == nbytes:
                raise
            self._buf = self._make(nbytes)


_ws8_cache: dict = {}


def _workspace8(index: int, nbytes: int, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """The binding's own 8-bit workspace per device."""
    if index not in _ws8_cache:
        _ws8_cache[index] = GrowingWorkspace(functools.partial(make_fp8_workspace, torch.device("cuda", index)))
    return _ws8_cache[index].get(nbytes, stream)


def _check8(what, out, query, key_cache, value_cache, scales, block_tables, context_lens, S, index):
    NB, Hkv, B, d = key_cache.shape
    if query.shape[2] != d or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise ValueError(f"{what}: shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError(f"{what}: block_tables must be [S][max_blocks], context_lens [S]")
    if scales.shape != (NB, Hkv + Hkv % 2, 2):
        raise ValueError(f"{what}: scales must be [num_blocks][num_kv_heads rounded up to even][2]")
    f8, i32 = torch.float8_e4m3fn, torch.int32
    return (_at(out, "out", query.dtype, index), _at(query, "query", query.dtype, index),
            _at(key_cache, "key_cache", f8, index), _at(value_cache, "value_cache", f8, index),
            _at(scales, "scales", torch.float32, index), _at(block_tables, "block_tables", i32, index),
            _at(context_lens, "context_lens", i32, index))


def paged_attention_decode_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                               context_lens: torch.Tensor, scale: Optional[float] = None, max_context_len: int = 0,
                               partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """paged_attention_decode over an 8-bit cache (float8_e4m3fn caches and
    their block scales).  workspace from make_fp8_workspace, one call at a
    time; None takes the binding's own per-device buffer, which every 8-bit
    call without a workspace shares and which grows as they need (waiting for
    the device then; it cannot grow during a stream capture).  Returns out."""
    what = "paged_attention_decode_fp8"
    index = _cuda_index(query, "query")
    S, H, d = query.shape
    ptrs = _check8(what, out, query, key_cache, value_cache, scales, block_tables, context_lens, S, index)
    NB, Hkv, B, _ = key_cache.shape
    mb = block_tables.shape[1]
    if workspace is None:
        workspace = _workspace8(index, paged_attention_decode_fp8_workspace_size(
            S, H, Hkv, d, max_context_len if max_context_len > 0 else mb * B, partition_size), stream)
    _call(load().paged_attention_decode_fp8, what, index, *ptrs, S, mb, max_context_len, B, NB, H, Hkv, d,
          1.0 / math.sqrt(d) if scale is None else scale, partition_size, _at(workspace, "workspace", torch.uint8, index),
          workspace.numel(), _dtype_code(query), _raw_stream(stream, index))
    return out


def paged_attention_prefill_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                value_cache: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                                context_lens: torch.Tensor, query_start: torch.Tensor,
                                scale: Optional[float] = None, max_query_len: int = 0, max_context_len: int = 0,
                                workspace: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """paged_attention_prefill over an 8-bit cache.  max_context_len bounds the
    contexts (0: the whole table) and sizes the workspace, which holds that
    many tokens of every sequence in 16 bits.  workspace as for
    paged_attention_decode_fp8.  Returns out."""
    what = "paged_attention_prefill_fp8"
    index = _cuda_index(query, "query")
    T, H, d = query.shape
    S = context_lens.shape[0]
    ptrs = _check8(what, out, query, key_cache, value_cache, scales, block_tables, context_lens, S, index)
    if query_start.shape != (S + 1,):
        raise ValueError(f"{what}: query_start must be [S+1]")
    NB, Hkv, B, _ = key_cache.shape
    mb = block_tables.shape[1]
    if workspace is None:
        workspace = _workspace8(index, paged_attention_prefill_fp8_workspace_size(
            S, Hkv, d, B, max_context_len if max_context_len > 0 else mb * B), stream)
    _call(load().paged_attention_prefill_fp8, what, index, *ptrs, _at(query_start, "query_start", torch.int32, index), S,
          T, max_query_len, max_context_len, mb, B, NB, H, Hkv, d, 1.0 / math.sqrt(d) if scale is None else scale,
          _at(workspace, "workspace", torch.uint8, index), workspace.numel(), _dtype_code(query),
          _raw_stream(stream, index))
    return out


# -- sliding windows and shared prefixes ------------------------------------------------

def _check16(what, out, query, key_cache, value_cache, block_tables, context_lens, S):
    """The device, the six pointers, the table's width and the sizes [NB, Hkv, B] of a
    call over a 16-bit cache of S sequences."""
    qs, ks, bs = query.shape, key_cache.shape, block_tables.shape
    if len(qs) != 3 or len(ks) != 4 or qs[2] != ks[3] or out.shape != qs or value_cache.shape != ks:
        raise ValueError(f"{what}: shape mismatch")
    if len(bs) != 2 or bs[0] != S or context_lens.shape != (S,):
        raise ValueError(f"{what}: block_tables must be [S][max_blocks], context_lens [S]")
    index, dt, i32 = _cuda_index(query, "query"), query.dtype, torch.int32
    if not (out.get_device() == index and out.dtype is dt and out.is_contiguous() and query.is_contiguous()
            and key_cache.get_device() == index and key_cache.dtype is dt and key_cache.is_contiguous()
            and value_cache.get_device() == index and value_cache.dtype is dt and value_cache.is_contiguous()
            and block_tables.get_device() == index and block_tables.dtype is i32 and block_tables.is_contiguous()
            and context_lens.get_device() == index and context_lens.dtype is i32 and context_lens.is_contiguous()):
        for t, name, dtype in ((out, "out", dt), (query, "query", dt), (key_cache, "key_cache", dt),     # says what is wrong
                               (value_cache, "value_cache", dt), (block_tables, "block_tables", i32),
                               (context_lens, "context_lens", i32)):
            _at(t, name, dtype, index)
    return (index, (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                    block_tables.data_ptr(), context_lens.data_ptr()), bs[1], ks)


_MOST = 2 ** 31 - 1        # a window or number of sinks beyond every context, as the C calls take it


_scratches = threading.local()


def _scratch(index: int, nbytes: int, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Uninitialised scratch of one call.  Kept per thread and stream, where calls
    follow one another (two threads may interleave their launches on one stream);
    a captured call takes memory of its own, which its graph keeps."""
    if torch.cuda.current_device() != index:               # streams and captures are asked for on the current device
        with torch.cuda.device(index):
            return _scratch(index, nbytes, stream)
    key = (index, _raw_stream(stream, index))
    held = _scratches.__dict__
    buf = held.get(key)
    if buf is not None and buf.numel() >= nbytes and not (
            torch._C._cuda_isCurrentStreamCapturing() if stream is None else _capturing(stream)):
        return buf
    with _on(stream):
        buf = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=torch.device("cuda", index))
    if not _capturing(stream):
        held[key] = buf
    return buf


def _limits(what: str, window: int, num_sinks: int):
    if window < 1 or num_sinks < 0:
        raise ValueError(f"{what}: window {window} (at least 1), {num_sinks} sinks (at least 0)")
    return min(window, _MOST), min(num_sinks, _MOST)


def paged_attention_decode_window(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                  value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  window: int, num_sinks: int = 0, scale: Optional[float] = None,
                                  max_context_len: int = 0,
                                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """paged_attention_decode over the last `window` tokens of each context (the
    newest among them) and its first num_sinks ones.  Table entries of blocks
    without a visible token are not read.  No workspace; calls may overlap.
    Returns out."""
    what = "paged_attention_decode_window"
    if window > _MOST or num_sinks > _MOST or window < 1 or num_sinks < 0:
        window, num_sinks = _limits(what, window, num_sinks)
    S, H, d = query.shape
    index, ptrs, mb, (NB, Hkv, B, _) = _check16(what, out, query, key_cache, value_cache, block_tables, context_lens, S)
    _call(load().paged_attention_decode_window, what, index, *ptrs, S, mb, max_context_len, B, NB, H, Hkv, d,
          1.0 / math.sqrt(d) if scale is None else scale, window, num_sinks, _dtype_code(query), _raw_stream(stream, index))
    return out


def paged_attention_prefill_window(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                                   query_start: torch.Tensor, window: int, num_sinks: int = 0,
                                   scale: Optional[float] = None, max_query_len: int = 0,
                                   workspace: Optional[torch.Tensor] = None,
                                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """paged_attention_prefill in which the new token at position p sees the
    tokens after p - window up to itself and the first num_sinks ones.  workspace:
    from make_workspace (its counter balances the work over the SMs), one call at
    a time; None: each SM takes a fixed share, and calls may overlap.  Returns out."""
    what = "paged_attention_prefill_window"
    if window > _MOST or num_sinks > _MOST or window < 1 or num_sinks < 0:
        window, num_sinks = _limits(what, window, num_sinks)
    T, H, d = query.shape
    S = context_lens.shape[0]
    index, ptrs, mb, (NB, Hkv, B, _) = _check16(what, out, query, key_cache, value_cache, block_tables, context_lens, S)
    if query_start.shape != (S + 1,):
        raise ValueError(f"{what}: query_start must be [S+1]")
    ws = (None, 0) if workspace is None else (_at(workspace, "workspace", torch.uint8, index), workspace.numel())
    _call(load().paged_attention_prefill_window, what, index, *ptrs,
          _at(query_start, "query_start", torch.int32, index), S, T, max_query_len, mb, B, NB, H, Hkv, d,
          1.0 / math.sqrt(d) if scale is None else scale, window, num_sinks, *ws, _dtype_code(query),
          _raw_stream(stream, index))
    return out


def paged_attention_decode_shared_workspace_size(num_seqs: int, num_groups: int, num_heads: int, num_kv_heads: int,
                                                 head_dim: int, max_context_len: int, max_prefix_len: int = 0,
                                                 max_group_size: int = 0, max_suffix_len: int = 0,
                                                 device: Optional[int] = None) -> int:
    """Bytes of scratch of a call on GPU number `device` (None: the current one),
    whose SMs decide how the work is split."""
    sizes = (num_seqs, num_groups, num_heads, num_kv_heads, head_dim, max_context_len, max_prefix_len, max_group_size,
             max_suffix_len)
    if device is None and torch.cuda.is_initialized():
        device = torch.cuda.current_device()
    return _shared_size(*sizes) if device is None else _shared_size_on(device, *sizes)


def _shared_size(*sizes) -> int:
    return int(load().paged_attention_decode_shared_workspace_size(*sizes))


@functools.lru_cache(maxsize=4096)
def _shared_size_on(index: int, *sizes) -> int:
    """Kept per device: asked of the device the first time."""
    if torch.cuda.current_device() == index:
        return _shared_size(*sizes)
    with torch.cuda.device(index):
        return _shared_size(*sizes)


def paged_attention_decode_shared(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                  value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  group_start: torch.Tensor, prefix_lens: torch.Tensor,
                                  scale: Optional[float] = None, max_context_len: int = 0, max_prefix_len: int = 0,
                                  max_group_size: int = 0, max_suffix_len: int = 0,
                                  workspace: Optional[torch.Tensor] = None,
                                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """paged_attention_decode of groups of sequences that begin with the same
    blocks, which are read once for a group.  group_start int32 [G+1]: group g is
    the sequences from group_start[g] on; prefix_lens int32 [S]: how many of its
    first tokens a sequence shares with its group, which are read through the
    table of the group's first sequence.  The max_* bounds (0: as large as the
    batch allows) size the workspace and the split of the work.  workspace: uint8
    scratch of paged_attention_decode_shared_workspace_size bytes, in no
    particular state, for one call at a time; None takes the binding's own, kept
    for the calling thread and stream.  Returns out."""
    what = "paged_attention_decode_shared"
    S, H, d = query.shape
    index, ptrs, mb, (NB, Hkv, B, _) = _check16(what, out, query, key_cache, value_cache, block_tables, context_lens, S)
    if group_start.dim() != 1 or not group_start.shape[0] or prefix_lens.shape != (S,):
        raise ValueError(f"{what}: group_start must be [G+1], prefix_lens [S]")
    G = group_start.shape[0] - 1
    if workspace is None:
        need = _shared_size_on(index, S, G, H, Hkv, d, max_context_len or mb * B, max_prefix_len, max_group_size, max_suffix_len)
        workspace = _scratch(index, need, stream)
    _call(load().paged_attention_decode_shared, what, index, *ptrs, _at(group_start, "group_start", torch.int32, index),
          _at(prefix_lens, "prefix_lens", torch.int32, index), S, G, max_group_size, max_prefix_len, max_suffix_len, mb,
          max_context_len, B, NB, H, Hkv, d, 1.0 / math.sqrt(d) if scale is None else scale,
          _at(workspace, "workspace", torch.uint8, index), workspace.numel(), _dtype_code(query),
          _raw_stream(stream, index))
    return out


def copy_blocks(cache: torch.Tensor, src_dst_pairs: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """cache [NB][...] (one block per leading index); src_dst_pairs int32 [n][2] on the device."""
    n = src_dst_pairs.shape[0] if src_dst_pairs.dim() == 2 else 0
    if src_dst_pairs.numel() and (src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2):
        raise ValueError("copy_blocks: src_dst_pairs must be [n][2]")
    NB = cache.shape[0]
    block_bytes = (cache.numel() // NB if NB else 0) * cache.element_size()
    pairs_ptr = _dev(src_dst_pairs, "src_dst_pairs", torch.int32) if n else None
    rc = load().copy_blocks(_dev(cache, "cache"), pairs_ptr, n, block_bytes, NB, _stream(stream, cache.device))
    _ck(rc, "copy_blocks")


def validate_copy_pairs(pairs, num_blocks: int) -> None:
    """Host-side check: ids in range, distinct destinations, no destination
    that is also a source.  Raises PkvError (PKV_EINVAL) otherwise."""
    a = np.ascontiguousarray(np.asarray(pairs, dtype=np.int32).reshape(-1, 2))
    rc = load().pkv_validate_copy_pairs(a.ctypes.data_as(ctypes.c_void_p) if a.size else None,
                                        a.shape[0], num_blocks)
    _ck(rc, "validate_copy_pairs")


def swap_blocks(dst_pool: torch.Tensor, src_pool: torch.Tensor, pairs: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Block pairs[p][1] of dst_pool takes block pairs[p][0] of src_pool (one
    launch for all pairs).  Pools [NB][...] of one layout: CUDA tensors or
    pinned host tensors; pairs int32 [n][2] on the GPU or pinned."""
    def addr(t, name):
        if not isinstance(t, torch.Tensor) or not (t.is_cuda or t.is_pinned()):
            raise TypeError(f"{name} must be a CUDA tensor or pinned host memory")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()
    if dst_pool.shape[1:] != src_pool.shape[1:] or dst_pool.dtype != src_pool.dtype:
        raise ValueError("swap_blocks: pools of different layouts")
    n = pairs.shape[0] if pairs.dim() == 2 else 0
    if n == 0:
        return
    if pairs.dtype != torch.int32 or pairs.shape[1] != 2:
        raise TypeError("swap_blocks: pairs must be int32 [n][2]")
    block_bytes = dst_pool[0].numel() * dst_pool.element_size()
    dev = dst_pool.device if dst_pool.is_cuda else src_pool.device
    rc = load().swap_blocks(addr(dst_pool, "dst_pool"), addr(src_pool, "src_pool"), addr(pairs, "pairs"), n,
                            block_bytes, src_pool.shape[0], dst_pool.shape[0], _stream(stream, dev))
    _ck(rc, "swap_blocks")


_FLAG_TIMEOUT = 8          # kFlagTimeout of the device's status word


def check(stream: Optional[torch.cuda.Stream] = None, device=None) -> None:
    """Synchronise the stream and raise if the device latched an index error
    or a wait timeout since the last check.  After a timeout the workspaces made
    here (make_workspace, make_fp8_workspace, the bindings' and the engine's
    own) have been prepared again, once the device had finished its work."""
    s = stream if stream is not None else torch.cuda.current_stream(device)
    try:
        _ck(load().pkv_check(ctypes.c_void_p(s.cuda_stream)), "pkv_check")
    except PkvError as e:
        flags = re.search(r"device error flags 0x([0-9a-f]+)", str(e))
        if flags and int(flags[1], 16) & _FLAG_TIMEOUT:
            _prepare_again(torch.cuda.current_device())
        raise


# -- host block allocator ---------------------------------------------------------

class BlockAllocator:
    """The native ref-counted block allocator (fork / append / free)."""

    def __init__(self, num_blocks: int, block_size: int, free_order: Optional[Sequence[int]] = None):
        self._L = load()
        h = ctypes.c_void_p()
        if free_order is not None:
            fo = np.ascontiguousarray(np.asarray(free_order, dtype=np.int32))
            if fo.shape != (num_blocks,):
                raise ValueError("free_order must list every block once")
            fp = fo.ctypes.data_as(ctypes.c_void_p)
        else:
            fp = None
        _ck(self._L.pkv_alloc_create(num_blocks, block_size, fp, ctypes.byref(h)), "pkv_alloc_create")
        self._h = h
        self.num_blocks = num_blocks
        self.block_size = block_size

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._L.pkv_alloc_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    def seq_new(self, length: int) -> int:
        sid = ctypes.c_int32()
        _ck(self._L.pkv_seq_new(self._h, length, ctypes.byref(sid)), "pkv_seq_new")
        return sid.value

    def fork(self, seq: int) -> int:
        child = ctypes.c_int32()
        _ck(self._L.pkv_seq_fork(self._h, seq, ctypes.byref(child)), "pkv_seq_fork")
        return child.value

    def append(self, seq: int):
        """Returns (slot, cow) with cow = (src, dst) or None."""
        slot, src, dst = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        _ck(self._L.pkv_seq_append(self._h, seq, ctypes.byref(slot), ctypes.byref(src), ctypes.byref(dst)),
            "pkv_seq_append")
        return slot.value, (None if src.value < 0 else (src.value, dst.value))

    def append_batch(self, seqs: Sequence[int]):
        """One token per sequence, all or nothing.  Returns (slots int64[n], pairs int32[m][2])."""
        s = np.ascontiguousarray(np.asarray(seqs, dtype=np.int32))
        n = s.shape[0]
        slots = np.empty(n, np.int64)
        pairs = np.empty((max(n, 1), 2), np.int32)
        npairs = ctypes.c_int()
        _ck(self._L.pkv_seq_append_batch(self._h, s.ctypes.data_as(ctypes.c_void_p), n,
                                         slots.ctypes.data_as(ctypes.c_void_p),
                                         pairs.ctypes.data_as(ctypes.c_void_p), ctypes.byref(npairs)),
            "pkv_seq_append_batch")
        return slots, pairs[:npairs.value].copy()

    def free(self, seq: int) -> None:
        _ck(self._L.pkv_seq_free(self._h, seq), "pkv_seq_free")

    def seq_len(self, seq: int) -> int:
        n = ctypes.c_int64()
        _ck(self._L.pkv_seq_len(self._h, seq, ctypes.byref(n)), "pkv_seq_len")
        return n.value

    def block_table(self, seq: int) -> list:
        n = ctypes.c_int()
        self._L.pkv_seq_block_table(self._h, seq, None, 0, ctypes.byref(n))
        out = np.empty(max(n.value, 1), np.int32)
        _ck(self._L.pkv_seq_block_table(self._h, seq, out.ctypes.data_as(ctypes.c_void_p), out.shape[0],
                                        ctypes.byref(n)), "pkv_seq_block_table")
        return out[:n.value].tolist()

    def beam_step(self, beams: Sequence[int], parents: Sequence[int]):
        """One beam-search step: new candidate i continues beams[parents[i]]
        (the first child continues the sequence, later ones fork it; all
        append a token; unchosen beams are freed).  Returns (new beam ids,
        slots int64 [kn], copy-on-write pairs int32 [m][2]); PkvOOM leaves
        everything unchanged."""
        b = np.ascontiguousarray(np.asarray(beams, dtype=np.int32))
        p = np.ascontiguousarray(np.asarray(parents, dtype=np.int32))
        kn = p.shape[0]
        new = np.empty(max(kn, 1), np.int32)
        slots = np.empty(max(kn, 1), np.int64)
        pairs = np.empty((max(kn, 1), 2), np.int32)
        npairs = ctypes.c_int()
        _ck(self._L.pkv_beam_step(self._h, b.ctypes.data_as(ctypes.c_void_p) if b.size else None, b.shape[0],
                                  p.ctypes.data_as(ctypes.c_void_p) if kn else None, kn,
                                  new.ctypes.data_as(ctypes.c_void_p), slots.ctypes.data_as(ctypes.c_void_p),
                                  pairs.ctypes.data_as(ctypes.c_void_p), ctypes.byref(npairs)), "pkv_beam_step")
        return new[:kn].tolist(), slots[:kn].copy(), pairs[:npairs.value].copy()

    def blocks_in_use(self) -> int:
        return self._L.pkv_blocks_in_use(self._h)

    def move_group(self, dst: "BlockAllocator", seqs: Sequence[int]):
        """Move the sequence group `seqs` (holding every reference to its
        blocks) to allocator `dst`, all or nothing: returns (new ids in dst,
        pairs int32 [m][2] of (block here, block in dst)) for swap_blocks.
        PkvOOM if dst has too few free blocks."""
        s = np.ascontiguousarray(np.asarray(seqs, dtype=np.int32))
        n = s.shape[0]
        ids = np.empty(max(n, 1), np.int32)
        cap = max(1, sum(len(self.block_table(int(x))) for x in s))
        pairs = np.empty((cap, 2), np.int32)
        npairs = ctypes.c_int()
        _ck(self._L.pkv_move_group(self._h, dst._h, s.ctypes.data_as(ctypes.c_void_p) if n else None, n,
                                   ids.ctypes.data_as(ctypes.c_void_p), pairs.ctypes.data_as(ctypes.c_void_p), cap,
                                   ctypes.byref(npairs)), "pkv_move_group")
        return ids[:n].tolist(), pairs[:npairs.value].copy()

    def build_block_tables(self, seqs: Sequence[int], max_blocks: int):
        """(tables int32 [n][max_blocks] padded with -1, context_lens int32 [n])."""
        s = np.ascontiguousarray(np.asarray(seqs, dtype=np.int32))
        n = s.shape[0]
        tables = np.empty((n, max_blocks), np.int32)
        ctx = np.empty(n, np.int32)
        _ck(self._L.pkv_build_block_tables(self._h, s.ctypes.data_as(ctypes.c_void_p), n,
                                           tables.ctypes.data_as(ctypes.c_void_p), max_blocks,
                                           ctx.ctypes.data_as(ctypes.c_void_p)), "pkv_build_block_tables")
        return tables, ctx

    def block_ref(self, block: int) -> int:
        return self._L.pkv_block_ref(self._h, block)

    def num_free(self) -> int:
        return self._L.pkv_num_free(self._h)

    def free_list(self) -> list:
        n = ctypes.c_int()
        out = np.empty(max(self.num_blocks, 1), np.int32)
        _ck(self._L.pkv_free_list(self._h, out.ctypes.data_as(ctypes.c_void_p), out.shape[0], ctypes.byref(n)),
            "pkv_free_list")
        return out[:n.value].tolist()
