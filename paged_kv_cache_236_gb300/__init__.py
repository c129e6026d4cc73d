"""Attention over a block-paged KV cache on GB300 (sm_103a).

A thin ctypes binding over the C ABI of ``libpaged_kv.so`` (declared in
``include/paged_kv.h``): argument marshalling only - every step of the path
runs in the library's CUDA kernels.  PyTorch supplies device memory and the
current stream.  There is no CPU fallback: if the library is missing or the
tensors are not on a CUDA device, the calls raise.

    paged_kv_write(k, v, slot_mapping, k_cache, v_cache)
    paged_attention_forward(q, k_cache, v_cache, block_tables, context_lens,
                            query_start_loc, scale, causal)
    paged_kv_write_fp8(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale)
    paged_attention_forward_fp8kv(q, k_cache, v_cache, ..., scale, k_scale, v_scale)
    BlockManager(num_blocks, block_size, max_blocks_per_seq)   (host, C++)
    copy_blocks(k_cache, v_cache, copies)                      (copy-on-write)
    paged_kv_write_rope(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache)
    paged_attention_scores(q, k_cache, block_tables, ..., scores, scale)
    paged_kv_select(scores, context_lens, budget)
    paged_kv_compact(k_cache, v_cache, block_tables, kept)     (eviction)

Block pool per layer: ``[num_blocks, block_size, num_kv_heads, head_dim]``
("ADR 004: Paged Attention Serving Integration", Decision 4 - a per-layer
cache tensor; "Paged Attention 基础", section 2 - fixed-size physical
blocks named by block tables).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import numpy as np
import torch

__all__ = [
    "paged_kv_write", "paged_attention_forward", "workspace_size", "workspace_min",
    "device_errors", "debug_fault", "set_profile_events", "set_profile_mid_event", "profile_elapsed_ms", "lib", "LibraryError", "DEVERR",
    "BlockManager", "OutOfBlocks", "copy_blocks", "paged_kv_write_fp8", "paged_attention_forward_fp8kv",
    "paged_kv_write_attention_forward", "paged_kv_write_attention_forward_fp8kv",
    "paged_kv_write_rope", "paged_kv_write_rope_fp8", "rope_frequencies", "rope_amplitude",
    "paged_attention_scores", "paged_attention_scores_fp8kv", "scores_workspace_size", "scores_workspace_min",
    "paged_kv_select", "paged_kv_compact",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpaged_kv.so")

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA, PKV_ERR_WORKSPACE, PKV_ERR_OUT_OF_BLOCKS = range(6)
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
HINT_SHARED_PREFIX = 0x1  # PKV_HINT_SHARED_PREFIX
DEVERR = {
    "slot_out_of_range": 0x1,
    "block_out_of_range": 0x2,
    "bad_sequence": 0x4,
    "timeout": 0x8,
    "plan_overflow": 0x10,
    "internal": 0x20,
}


class LibraryError(RuntimeError):
    """A non-OK status from the C ABI."""

    def __init__(self, status: int, message: str):
        super().__init__(f"paged_kv status {status}: {message}")
        self.status = status


class OutOfBlocks(LibraryError):
    """The block manager's free and evictable blocks do not cover a request
    (``PKV_ERR_OUT_OF_BLOCKS``); the manager is unchanged."""


_lib = None
_lock = threading.Lock()

c_vp, c_i32, c_i64, c_sz, c_f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_ROPE_ARGS = [c_vp] * 9 + [c_i64, c_i64] + [c_i32] * 6 + [c_f, c_i64, c_i64, c_i64, c_i32]
_SCORES_ARGS = [c_vp] * 8 + [c_i32, c_i64, c_i32, c_i32, c_i32, c_i64] + [c_i32] * 5 + [c_f, c_i32, c_f]


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_236_gb300.build` "
                    "(there is no CPU fallback)")
            L = ctypes.CDLL(LIB_PATH)
            L.paged_kv_write.restype = c_i32
            L.paged_kv_write.argtypes = [c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i32, c_i32, c_i32,
                                         c_i64, c_i64, c_i32, c_vp]
            L.paged_attention_workspace_size.restype = c_sz
            L.paged_attention_workspace_size.argtypes = [c_i32, c_i64, c_i32, c_i32, c_i32]
            L.paged_attention_workspace_min.restype = c_sz
            L.paged_attention_workspace_min.argtypes = [c_i32, c_i64, c_i32, c_i32, c_i32]
            L.paged_attention_forward.restype = c_i32
            L.paged_attention_forward.argtypes = [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i64, c_i32,
                                                  c_i32, c_i32, c_i64, c_i32, c_i32, c_i32, c_f, c_i32, c_i32,
                                                  c_vp, c_sz, c_i32, c_vp]
            L.pkv_last_error.restype = ctypes.c_char_p
            L.pkv_last_error.argtypes = []
            L.pkv_device_errors.restype = c_i32
            L.pkv_device_errors.argtypes = [ctypes.POINTER(c_i32), c_i32]
            L.pkv_set_profile_events.restype = None
            L.pkv_set_profile_events.argtypes = [c_vp, c_vp]
            L.pkv_set_profile_mid_event.restype = None
            L.pkv_set_profile_mid_event.argtypes = [c_vp]
            L.pkv_event_elapsed_ms.restype = c_i32
            L.pkv_event_elapsed_ms.argtypes = [c_vp, c_vp, ctypes.POINTER(c_f)]
            L.pkv_version.restype = ctypes.c_char_p
            L.pkv_version.argtypes = []
            for name, args in (("pkv_capture_id", [c_vp, ctypes.POINTER(ctypes.c_uint64)]),
                               ("pkv_capture_watch", [c_vp]),
                               ("pkv_capture_gone", [ctypes.POINTER(ctypes.c_uint64)])):
                getattr(L, name).restype = c_i32
                getattr(L, name).argtypes = args
            L.pkv_debug_fault.restype = c_i32
            L.pkv_debug_fault.argtypes = [c_i32, c_i64]
            L.paged_kv_write_attention_forward.restype = c_i32
            L.paged_kv_write_attention_forward.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64] + \
                L.paged_attention_forward.argtypes
            L.paged_kv_write_attention_forward_fp8kv.restype = c_i32
            L.paged_kv_write_attention_forward_fp8kv.argtypes = [
                c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i64,
                c_i32, c_i32, c_i32, c_i64, c_i32, c_i32, c_i32, c_f, c_i32, c_f, c_f, c_i32, c_vp, c_sz, c_vp]
            c_p32 = ctypes.POINTER(c_i32)
            for name, args in (
                    ("pkv_bm_create", [c_i32, c_i32, c_i32, ctypes.POINTER(c_vp)]),
                    ("pkv_bm_update", [c_vp, c_i64, c_i32, c_vp, c_p32, c_p32]),
                    ("pkv_bm_step", [c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_p32]),
                    ("pkv_bm_free", [c_vp, c_i64]),
                    ("pkv_bm_fork", [c_vp, c_i64, c_i64]),
                    ("pkv_bm_compact", [c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp]),
                    ("pkv_bm_add_prefix", [c_vp, c_i64, c_vp, c_i32]),
                    ("pkv_bm_try_get_prefix_blocks", [c_vp, c_i64, c_vp, c_i32, c_p32]),
                    ("pkv_bm_block_table", [c_vp, c_i64, c_vp, c_p32, c_p32]),
                    ("pkv_bm_stats", [c_vp, c_p32, c_p32, c_p32, c_p32]),
                    ("paged_kv_copy_blocks", [c_vp, c_vp, c_vp, c_i32, c_i32, c_i64, c_i64, c_i32, c_i32, c_i32,
                                              c_i32, c_vp]),
                    ("paged_kv_write_fp8", [c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i32, c_i32, c_i32, c_i64,
                                            c_i64, c_i32, c_f, c_f, c_vp]),
                    ("paged_attention_forward_fp8kv", [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i64, c_i32,
                                                       c_i32, c_i32, c_i64, c_i32, c_i32, c_i32, c_f, c_i32, c_f,
                                                       c_f, c_i32, c_vp, c_sz, c_vp]),
                    ("paged_kv_write_rope", _ROPE_ARGS + [c_vp]),
                    ("paged_kv_write_rope_fp8", _ROPE_ARGS + [c_f, c_f, c_vp]),
                    ("paged_attention_scores", _SCORES_ARGS + [c_vp, c_sz, c_i32, c_vp]),
                    ("paged_attention_scores_fp8kv", _SCORES_ARGS + [c_f, c_vp, c_sz, c_vp]),
                    ("paged_kv_select", [c_vp] * 4 + [c_i32] * 7 + [c_vp]),
                    ("paged_kv_compact", [c_vp] * 7 + [c_i32] * 3 + [c_i64] + [c_i32] * 6 + [c_vp])):
                getattr(L, name).restype = c_i32
                getattr(L, name).argtypes = args
            for name in ("paged_attention_scores_workspace_size", "paged_attention_scores_workspace_min"):
                getattr(L, name).restype = c_sz
                getattr(L, name).argtypes = [c_i32, c_i64, c_i32, c_i32, c_i64]
            L.pkv_bm_destroy.restype = None
            L.pkv_bm_destroy.argtypes = [c_vp]
            _lib = L
    return _lib


def _check(status: int) -> None:
    if status != PKV_OK:
        msg = lib().pkv_last_error().decode(errors="replace")
        raise (OutOfBlocks if status == PKV_ERR_OUT_OF_BLOCKS else LibraryError)(status, msg)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    if _raw_stream and device.index is not None:  # a microsecond less than through a stream object
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need_cuda(*tensors: torch.Tensor) -> torch.device:
    dev = tensors[0].device
    for t in tensors:
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
            raise ValueError("all tensors must be CUDA tensors (no CPU path)")
        if t.device != dev:
            raise ValueError("all tensors must be on the same device")
    return dev


def paged_kv_write(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor) -> None:
    """Scatter ``k, v [T, Hkv, D]`` into ``k_cache, v_cache [NB, bs, Hkv, D]``
    at ``slot_mapping [T]`` (int64; slot = block * bs + offset; < 0 skips)."""
    dev = _need_cuda(k, v, slot_mapping, k_cache, v_cache)
    if k_cache.dtype not in DTYPE or k.dtype != k_cache.dtype or v.dtype != k_cache.dtype or \
            v_cache.dtype != k_cache.dtype:
        raise ValueError("k, v, k_cache, v_cache must share dtype bfloat16 or float32")
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() or \
            not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, num_kv_heads, head_dim]")
    NB, bs, Hkv, D = k_cache.shape
    T = k.shape[0]
    for name, t in (("k", k), ("v", v)):
        if t.dim() != 3 or tuple(t.shape[1:]) != (Hkv, D) or t.stride(2) != 1 or t.stride(1) != D:
            raise ValueError(f"{name} must be [T, {Hkv}, {D}] with contiguous heads")
    if v.shape[0] != T or slot_mapping.shape != (T,) or slot_mapping.dtype != torch.int64 or \
            not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous int64 [T]")
    with torch.cuda.device(dev):
        _check(lib().paged_kv_write(k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(),
                                    v_cache.data_ptr(), T, NB, bs, Hkv, D, k.stride(0) if T else 0,
                                    v.stride(0) if T else 0, DTYPE[k_cache.dtype], _stream(dev)))


def workspace_size(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().paged_attention_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim))


def workspace_min(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().paged_attention_workspace_min(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim))


class _Scratch(threading.local):
    """A thread's cached workspaces, per (device, stream).  A call is several
    launches that pass its plan through the workspace, and it runs without the
    interpreter's lock: two threads on one stream would put their launches
    between one another's.  They go with the thread."""

    def __init__(self):
        self.buffers: dict = {}
        self.pooled = 0  # id of a capture whose allocations a graph's memory pool serves


_scratch = _Scratch()
_graphs_hold: dict = {}  # capture id -> {stream: its workspaces, the one in use last}
_graphs_lock = threading.Lock()


def _workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    """Workspace of a call on dev's current stream (dev is the current device)."""
    if torch.cuda.is_current_stream_capturing():
        return _graph_workspace(dev, nbytes)
    key = (dev.index, _stream(dev))
    ws = _scratch.buffers.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
        _scratch.buffers[key] = ws
    return ws


def _graph_workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    """Workspace of a call that is being captured: the graph's own.  A cached
    one is replaced when a later call wants more, and graphs captured on one
    stream may be replayed on two.

    Under ``torch.cuda.graph`` an allocation comes from the graph's memory
    pool, which lasts as long as the graph.  Under any other capture it comes
    from the memory all tensors share, so it is held here until the graph is
    gone: one for each stream of the capture, which runs its calls in order."""
    stream, found = _stream(dev), ctypes.c_uint64(0)
    _check(lib().pkv_capture_id(stream, ctypes.byref(found)))
    capture = found.value
    with _graphs_lock:
        _drop_graphs_gone()
        first = capture not in _graphs_hold
        if first and _scratch.pooled != capture and _in_graph_pool(torch.empty(1, dtype=torch.uint8, device=dev)):
            _scratch.pooled = capture
        if _scratch.pooled == capture:
            return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
        if first:
            _check(lib().pkv_capture_watch(stream))
        mine = _graphs_hold.setdefault(capture, {}).setdefault((dev.index, stream), [])
        if not mine or mine[-1].numel() < nbytes:
            mine.append(torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev))
        return mine[-1]


def _drop_graphs_gone() -> None:
    """Gives up the workspaces of graphs that no longer exist (the lock held)."""
    found = ctypes.c_uint64(0)
    while True:
        _check(lib().pkv_capture_gone(ctypes.byref(found)))
        if found.value == 0:
            return
        _graphs_hold.pop(found.value, None)


def _in_graph_pool(t: torch.Tensor) -> bool:
    """Whether t's memory, allocated under a capture, is the graph's: of a private
    pool of the allocator, or a node of the graph itself (cudaMallocAsync)."""
    backend = torch.cuda.get_allocator_backend()
    if backend != "native":  # which alone can say
        return backend == "cudaMallocAsync"
    for segment in torch.cuda.memory_snapshot():
        if 0 <= t.data_ptr() - segment["address"] < segment["total_size"]:
            return tuple(segment.get("segment_pool_id", (0, 0))) != (0, 0)
    return False


def paged_attention_forward(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, context_lens: torch.Tensor,
                            query_start_loc: torch.Tensor, scale: float, causal: bool = True, *,
                            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                            max_query_len: int = 0, shared_prefix: bool = False) -> torch.Tensor:
    """Varlen attention of ``q [T, Hq, D]`` through per-sequence block tables.

    ``context_lens[s]`` counts sequence s's tokens after this step's write
    (its query tokens included); query i of n sits at position L - n + i.
    ``workspace`` (uint8, >= ``workspace_min``) defaults to a cached buffer
    per (thread, device, stream).  ``max_query_len`` is an optional host hint.
    ``shared_prefix`` tells the call that consecutive sequences may start
    with the same physical blocks (prefix caching): runs of them then read
    their common prefix once (``PKV_HINT_SHARED_PREFIX``).
    """
    dev = _need_cuda(q, k_cache, v_cache, block_tables, context_lens, query_start_loc)
    args, out, workspace = _forward_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
                                         causal, out, workspace, max_query_len, shared_prefix, dev)
    with torch.cuda.device(dev):
        _check(lib().paged_attention_forward(*args))
    return out


def _forward_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale, causal, out, workspace,
                  max_query_len, shared_prefix, dev) -> tuple:
    """Checks paged_attention_forward's tensors; returns (its C arguments, out,
    the workspace, to be kept until the call has returned)."""
    if q.dtype not in DTYPE or k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise ValueError("q, k_cache, v_cache must share dtype bfloat16 or float32")
    if q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be contiguous [T, Hq, D]")
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() or \
            not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, num_kv_heads, head_dim]")
    T, Hq, D = q.shape
    NB, bs, Hkv, Dk = k_cache.shape
    if Dk != D:
        raise ValueError("head_dim of q and the caches differ")
    B = context_lens.shape[0]
    for name, t, shape in (("block_tables", block_tables, None), ("context_lens", context_lens, (B,)),
                           ("query_start_loc", query_start_loc, (B + 1,))):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
        if shape is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or (B > 0 and block_tables.shape[1] == 0):
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq] with max_blocks_per_seq > 0")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must match q")
    with torch.cuda.device(dev):
        need = workspace_min(B, T, Hq, Hkv, D)
        if workspace is None:
            workspace = _workspace(dev, workspace_size(B, T, Hq, Hkv, D))
        if workspace.dtype != torch.uint8 or workspace.device != dev or workspace.numel() < need:
            raise ValueError(f"workspace must be a uint8 CUDA tensor of at least {need} bytes")
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            query_start_loc.data_ptr(), out.data_ptr(), B, T, Hq, Hkv, D, NB, bs, max(1, block_tables.shape[1]),
            int(max_query_len), float(scale), 1 if causal else 0, HINT_SHARED_PREFIX if shared_prefix else 0,
            workspace.data_ptr(), workspace.numel(), DTYPE[q.dtype], _stream(dev))
    return args, out, workspace


def _new_rows(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, Hkv: int, D: int, dtypes) -> tuple:
    """Checks a step's new K/V rows [T, Hkv, D] (contiguous heads) and returns
    (T, k token stride, v token stride)."""
    if k.dtype not in dtypes or v.dtype != k.dtype:
        raise ValueError("k and v must share a dtype the pools accept")
    T = k.shape[0]
    for name, t in (("k", k), ("v", v)):
        if t.dim() != 3 or tuple(t.shape[1:]) != (Hkv, D) or t.stride(2) != 1 or t.stride(1) != D:
            raise ValueError(f"{name} must be [T, {Hkv}, {D}] with contiguous heads")
    if v.shape[0] != T or slot_mapping.shape != (T,) or slot_mapping.dtype != torch.int64 or \
            not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous int64 [T]")
    return T, (k.stride(0) if T else 0), (v.stride(0) if T else 0)


def paged_kv_write_attention_forward(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                                     q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                     block_tables: torch.Tensor, context_lens: torch.Tensor,
                                     query_start_loc: torch.Tensor, scale: float, causal: bool = True, *,
                                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                     max_query_len: int = 0, shared_prefix: bool = False) -> torch.Tensor:
    """``paged_kv_write(k, v, slot_mapping, k_cache, v_cache)`` then
    ``paged_attention_forward(q, k_cache, v_cache, ...)`` in one call: the
    new rows are written by extra CTAs of the planner's launch (one launch
    fewer per step).  Same arguments and result as the two calls."""
    dev = _need_cuda(k, v, slot_mapping, q, k_cache, v_cache, block_tables, context_lens, query_start_loc)
    Tn, ks, vs = _new_rows(k, v, slot_mapping, k_cache.shape[2], k_cache.shape[3], {k_cache.dtype})
    args, out, workspace = _forward_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
                                         causal, out, workspace, max_query_len, shared_prefix, dev)
    with torch.cuda.device(dev):
        _check(lib().paged_kv_write_attention_forward(k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), Tn, ks, vs,
                                                      *args))
    return out


def set_profile_events(start, stop) -> None:
    """Record ``start``/``stop`` (torch.cuda.Event) around the attention
    kernels of later forward calls on this thread; ``None, None`` stops."""
    if start is None or stop is None:
        lib().pkv_set_profile_events(None, None)
    else:
        lib().pkv_set_profile_events(start.cuda_event, stop.cuda_event)


def set_profile_mid_event(mid) -> None:
    """Also record ``mid`` (torch.cuda.Event) right after the multi-token
    tensor-core kernel of later forward calls on this thread; ``None`` stops."""
    lib().pkv_set_profile_mid_event(None if mid is None else mid.cuda_event)


def profile_elapsed_ms(start, stop) -> float:
    """Milliseconds between two events recorded through ``set_profile_events``."""
    ms = c_f(0.0)
    _check(lib().pkv_event_elapsed_ms(start.cuda_event, stop.cuda_event, ctypes.byref(ms)))
    return float(ms.value)


def debug_fault(fault_tile: int, wait_ns: int) -> None:
    """Testing hook (``pkv_debug_fault``): arm the next forward or scores
    call of this thread to give up its waits after ``wait_ns`` ns and, with
    ``fault_tile`` >= 1, to skip the loads of one tile in one CTA, so that the
    bounded waits run out."""
    _check(lib().pkv_debug_fault(int(fault_tile), int(wait_ns)))


def device_errors(clear: bool = True) -> int:
    """Sticky device error bits (``DEVERR``) of the current device; synchronises."""
    flags = c_i32(0)
    _check(lib().pkv_device_errors(ctypes.byref(flags), 1 if clear else 0))
    return int(flags.value)


# ----------------------------------------------------------------------------
# host block manager (include/paged_kv_blocks.h)
# ----------------------------------------------------------------------------

def _host(a, dtype) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=dtype))


class BlockManager:
    """The library's host block manager: block ids, slots and tables for a
    pool of ``num_blocks`` blocks of ``block_size`` tokens ("Paged Attention
    基础", section 3.1 C; "ADR 004", Decision 5 and Consequences).

    ``update(seq, n)`` -> (slots int64 [n], copies int32 [c, 2]);
    ``step(seq_ids, n_new)`` -> dict of the call metadata (host numpy
    arrays: slot_mapping, block_tables, context_lens, query_start_loc,
    copies); ``compact``, ``free``, ``fork``, ``add_prefix``,
    ``try_get_prefix_blocks``, ``block_table``, ``stats``.  Refused requests raise ``OutOfBlocks`` or
    ``LibraryError`` and change nothing.
    """

    def __init__(self, num_blocks: int, block_size: int, max_blocks_per_seq: int):
        h = c_vp()
        _check(lib().pkv_bm_create(num_blocks, block_size, max_blocks_per_seq, ctypes.byref(h)))
        self._h = h
        self.num_blocks, self.block_size, self.max_blocks = num_blocks, block_size, max_blocks_per_seq

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            try:
                _lib.pkv_bm_destroy(h)
            except Exception:  # interpreter shutdown: the library may be gone already
                pass
            self._h = None

    def update(self, seq: int, n: int):
        slots = np.empty(max(n, 0), dtype=np.int64)
        pair = (c_i32 * 2)()
        nc = c_i32(0)
        _check(lib().pkv_bm_update(self._h, int(seq), int(n), slots.ctypes.data if n > 0 else None, pair,
                                   ctypes.byref(nc)))
        return slots, np.asarray(list(pair)[:2 * nc.value], dtype=np.int32).reshape(-1, 2)

    def step(self, seq_ids, n_new, reuse: bool = False) -> dict:
        """One batch step (``pkv_bm_step``): the call metadata as host numpy
        arrays.  With ``reuse=True`` they are views into buffers the manager
        keeps, valid until its next ``step(..., reuse=True)``; this saves the
        per-call allocations of a serving loop."""
        ids = _host(seq_ids, np.int64)
        n = _host(n_new, np.int32)
        B = len(ids)
        if len(n) != B:
            raise ValueError("seq_ids and n_new differ in length")
        total = int(n.sum(dtype=np.int64)) if B else 0
        if reuse:
            bufs = self._buffers(B, total)
            out = {k: v for k, v in bufs["arrays"].items()}
            ptr = bufs["ptr"]
            nc = bufs["nc"]
            _check(lib().pkv_bm_step(self._h, ids.ctypes.data if B else None, n.ctypes.data if B else None, B,
                                     ptr["slot_mapping"], ptr["block_tables"], ptr["context_lens"],
                                     ptr["query_start_loc"], ptr["copies"], ctypes.byref(nc)))
            return {"slot_mapping": out["slot_mapping"][:total], "block_tables": out["block_tables"][:B],
                    "context_lens": out["context_lens"][:B], "query_start_loc": out["query_start_loc"][:B + 1],
                    "copies": out["copies"][:nc.value]}
        out = {
            "slot_mapping": np.empty(max(total, 0), dtype=np.int64),
            "block_tables": np.empty((B, self.max_blocks), dtype=np.int32),
            "context_lens": np.empty(B, dtype=np.int32),
            "query_start_loc": np.empty(B + 1, dtype=np.int32),
            "copies": np.empty((max(B, 1), 2), dtype=np.int32),
        }
        nc = c_i32(0)
        ptr = lambda a: a.ctypes.data if a.size else None
        _check(lib().pkv_bm_step(self._h, ptr(ids), ptr(n), B, ptr(out["slot_mapping"]), ptr(out["block_tables"]),
                                 ptr(out["context_lens"]), out["query_start_loc"].ctypes.data,
                                 out["copies"].ctypes.data, ctypes.byref(nc)))
        out["copies"] = out["copies"][:nc.value]
        return out

    def _buffers(self, B: int, total: int) -> dict:
        """Output buffers of at least B sequences and `total` new tokens,
        grown geometrically, with their addresses computed once."""
        b = getattr(self, "_bufs", None)
        if b is None or b["B"] < B or b["T"] < total:
            cb = max(B, 2 * b["B"] if b else 64, 1)
            ct = max(total, 2 * b["T"] if b else 256, 1)
            arrays = {
                "slot_mapping": np.empty(ct, dtype=np.int64),
                "block_tables": np.empty((cb, self.max_blocks), dtype=np.int32),
                "context_lens": np.empty(cb, dtype=np.int32),
                "query_start_loc": np.empty(cb + 1, dtype=np.int32),
                "copies": np.empty((cb, 2), dtype=np.int32),
            }
            b = {"B": cb, "T": ct, "arrays": arrays, "nc": c_i32(0),
                 "ptr": {k: a.ctypes.data for k, a in arrays.items()}}
            self._bufs = b
        return b

    def free(self, seq: int) -> None:
        _check(lib().pkv_bm_free(self._h, int(seq)))

    def fork(self, parent: int, child: int) -> None:
        _check(lib().pkv_bm_fork(self._h, int(parent), int(child)))

    def compact(self, seq_ids, num_tokens) -> dict:
        """Shorten sequences to at most ``num_tokens`` (an int, or one for
        each), as ``paged_kv_compact`` rewrites their caches: host arrays
        ``block_tables`` and ``dst_block_tables`` (before and after, its two
        tables) and ``context_lens`` (after).  Blocks past the new lengths are
        given back; shared or cached blocks are replaced by new ones."""
        ids = _host(seq_ids, np.int64)
        B = len(ids)
        n = np.full(B, num_tokens, dtype=np.int32) if np.ndim(num_tokens) == 0 else _host(num_tokens, np.int32)
        if len(n) != B:
            raise ValueError("seq_ids and num_tokens differ in length")
        out = {"block_tables": np.empty((B, self.max_blocks), dtype=np.int32),
               "dst_block_tables": np.empty((B, self.max_blocks), dtype=np.int32),
               "context_lens": np.empty(B, dtype=np.int32)}
        ptr = lambda a: a.ctypes.data if a.size else None
        _check(lib().pkv_bm_compact(self._h, ptr(ids), ptr(n), B, ptr(out["block_tables"]),
                                    ptr(out["dst_block_tables"]), ptr(out["context_lens"])))
        return out

    def add_prefix(self, seq: int, tokens) -> None:
        t = _host(tokens, np.int64)
        _check(lib().pkv_bm_add_prefix(self._h, int(seq), t.ctypes.data if t.size else None, len(t)))

    def try_get_prefix_blocks(self, seq: int, tokens) -> int:
        t = _host(tokens, np.int64)
        got = c_i32(0)
        _check(lib().pkv_bm_try_get_prefix_blocks(self._h, int(seq), t.ctypes.data if t.size else None, len(t),
                                                  ctypes.byref(got)))
        return int(got.value)

    def block_table(self, seq: int) -> list:
        table = np.empty(self.max_blocks, dtype=np.int32)
        nb, nt = c_i32(0), c_i32(0)
        _check(lib().pkv_bm_block_table(self._h, int(seq), table.ctypes.data, ctypes.byref(nb), ctypes.byref(nt)))
        return table[:nb.value].tolist()

    def num_tokens(self, seq: int) -> int:
        nt = c_i32(0)
        _check(lib().pkv_bm_block_table(self._h, int(seq), None, None, ctypes.byref(nt)))
        return int(nt.value)

    def stats(self) -> dict:
        f, i, u, c = c_i32(0), c_i32(0), c_i32(0), c_i32(0)
        _check(lib().pkv_bm_stats(self._h, ctypes.byref(f), ctypes.byref(i), ctypes.byref(u), ctypes.byref(c)))
        return {"free": f.value, "idle": i.value, "in_use": u.value, "cached": c.value}


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, copies) -> None:
    """Copy-on-write on the device pool: block ``dst`` of every layer's K and
    V pool becomes a copy of block ``src`` for each host pair (src, dst) of
    ``copies`` (int32 [n, 2], as ``BlockManager.update`` / ``step`` return).
    Caches are ``[NB, bs, Hkv, D]`` or ``[layers, NB, bs, Hkv, D]`` (each
    layer's pool contiguous).  Runs on the current stream."""
    dev = _need_cuda(k_cache, v_cache)
    pairs = _host(copies, np.int32).reshape(-1, 2)
    if k_cache.dtype not in DTYPE or v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape or \
            v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache must share dtype (bfloat16 or float32), shape and strides")
    if k_cache.dim() == 4:
        layers, stride = 1, 0
        pool = k_cache
    elif k_cache.dim() == 5:
        layers, stride = k_cache.shape[0], k_cache.stride(0)
        pool = k_cache[0]
    else:
        raise ValueError("caches must be [NB, bs, Hkv, D] or [layers, NB, bs, Hkv, D]")
    if not pool.is_contiguous():
        raise ValueError("each layer's pool must be contiguous")
    NB, bs, Hkv, D = pool.shape
    with torch.cuda.device(dev):
        _check(lib().paged_kv_copy_blocks(k_cache.data_ptr(), v_cache.data_ptr(),
                                          pairs.ctypes.data if len(pairs) else None, len(pairs), layers, stride,
                                          NB, bs, Hkv, D, DTYPE[k_cache.dtype], _stream(dev)))


# ----------------------------------------------------------------------------
# FP8 (E4M3) pools (include/paged_kv.h: paged_kv_write_fp8,
# paged_attention_forward_fp8kv)
# ----------------------------------------------------------------------------

_FP8_TYPES = {torch.uint8} | ({torch.float8_e4m3fn} if hasattr(torch, "float8_e4m3fn") else set())


def _check_fp8_pools(k_cache: torch.Tensor, v_cache: torch.Tensor) -> None:
    if k_cache.dtype not in _FP8_TYPES or v_cache.dtype != k_cache.dtype:
        raise ValueError("FP8 pools must be uint8 (E4M3 codes) or float8_e4m3fn tensors")
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() or \
            not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, num_kv_heads, head_dim]")


def paged_kv_write_fp8(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, k_scale: float, v_scale: float) -> None:
    """Encode ``k, v [T, Hkv, D]`` (bf16 or f32) as E4M3 codes of x / scale
    and scatter them into the FP8 pools at ``slot_mapping`` (< 0 skips)."""
    dev = _need_cuda(k, v, slot_mapping, k_cache, v_cache)
    _check_fp8_pools(k_cache, v_cache)
    if k.dtype not in DTYPE or v.dtype != k.dtype:
        raise ValueError("k and v must share dtype bfloat16 or float32")
    NB, bs, Hkv, D = k_cache.shape
    T = k.shape[0]
    for name, t in (("k", k), ("v", v)):
        if t.dim() != 3 or tuple(t.shape[1:]) != (Hkv, D) or t.stride(2) != 1 or t.stride(1) != D:
            raise ValueError(f"{name} must be [T, {Hkv}, {D}] with contiguous heads")
    if v.shape[0] != T or slot_mapping.shape != (T,) or slot_mapping.dtype != torch.int64 or \
            not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous int64 [T]")
    with torch.cuda.device(dev):
        _check(lib().paged_kv_write_fp8(k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(),
                                        v_cache.data_ptr(), T, NB, bs, Hkv, D, k.stride(0) if T else 0,
                                        v.stride(0) if T else 0, DTYPE[k.dtype], float(k_scale), float(v_scale),
                                        _stream(dev)))


def paged_attention_forward_fp8kv(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  query_start_loc: torch.Tensor, scale: float, k_scale: float, v_scale: float,
                                  causal: bool = True, *, out: torch.Tensor | None = None,
                                  workspace: torch.Tensor | None = None, max_query_len: int = 0) -> torch.Tensor:
    """``paged_attention_forward`` over FP8 pools read as code * k_scale and
    code * v_scale; q and the result are bf16, head_dim 128."""
    dev = _need_cuda(q, k_cache, v_cache, block_tables, context_lens, query_start_loc)
    args, out, workspace = _fp8_forward_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
                                             k_scale, v_scale, causal, out, workspace, max_query_len, dev)
    with torch.cuda.device(dev):
        _check(lib().paged_attention_forward_fp8kv(*args))
    return out


def paged_kv_write_attention_forward_fp8kv(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                                           q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                           block_tables: torch.Tensor, context_lens: torch.Tensor,
                                           query_start_loc: torch.Tensor, scale: float, k_scale: float,
                                           v_scale: float, causal: bool = True, *, out: torch.Tensor | None = None,
                                           workspace: torch.Tensor | None = None,
                                           max_query_len: int = 0) -> torch.Tensor:
    """``paged_kv_write_fp8`` of a step's new rows (bf16 or f32) then
    ``paged_attention_forward_fp8kv``, in one call (the rows are encoded by
    extra CTAs of the planner's launch)."""
    dev = _need_cuda(k, v, slot_mapping, q, k_cache, v_cache, block_tables, context_lens, query_start_loc)
    _check_fp8_pools(k_cache, v_cache)
    Tn, ks, vs = _new_rows(k, v, slot_mapping, k_cache.shape[2], k_cache.shape[3], set(DTYPE))
    args, out, workspace = _fp8_forward_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
                                             k_scale, v_scale, causal, out, workspace, max_query_len, dev)
    with torch.cuda.device(dev):
        _check(lib().paged_kv_write_attention_forward_fp8kv(k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), Tn,
                                                            ks, vs, DTYPE[k.dtype], *args))
    return out


def _fp8_forward_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale, k_scale, v_scale,
                      causal, out, workspace, max_query_len, dev) -> tuple:
    """Checks paged_attention_forward_fp8kv's tensors; returns (its C arguments,
    out, the workspace, to be kept until the call has returned)."""
    _check_fp8_pools(k_cache, v_cache)
    if q.dtype != torch.bfloat16 or q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be contiguous bfloat16 [T, Hq, D]")
    T, Hq, D = q.shape
    NB, bs, Hkv, Dk = k_cache.shape
    if Dk != D:
        raise ValueError("head_dim of q and the caches differ")
    B = context_lens.shape[0]
    for name, t, shape in (("block_tables", block_tables, None), ("context_lens", context_lens, (B,)),
                           ("query_start_loc", query_start_loc, (B + 1,))):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
        if shape is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or (B > 0 and block_tables.shape[1] == 0):
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq] with max_blocks_per_seq > 0")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must match q")
    with torch.cuda.device(dev):
        need = workspace_min(B, T, Hq, Hkv, D)
        if workspace is None:
            workspace = _workspace(dev, workspace_size(B, T, Hq, Hkv, D))
        if workspace.dtype != torch.uint8 or workspace.device != dev or workspace.numel() < need:
            raise ValueError(f"workspace must be a uint8 CUDA tensor of at least {need} bytes")
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            query_start_loc.data_ptr(), out.data_ptr(), B, T, Hq, Hkv, D, NB, bs, max(1, block_tables.shape[1]),
            int(max_query_len), float(scale), 1 if causal else 0, float(k_scale), float(v_scale), 0,
            workspace.data_ptr(), workspace.numel(), _stream(dev))
    return args, out, workspace


# ----------------------------------------------------------------------------
# rotary positions with the K/V write (include/paged_kv.h: paged_kv_write_rope)
# ----------------------------------------------------------------------------

def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original_max_position: int = 0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda") -> torch.Tensor:
    """Rotary frequencies, float64 ``[rotary_dim / 2]`` in radians per
    position: ``base ** (-2 i / rotary_dim)``, changed for contexts ``factor``
    times longer than the ``original_max_position`` a model was trained on:

    * ``None``: unchanged;
    * ``"linear"``: every frequency / factor (positions interpolated);
    * ``"ntk"``: base * factor ** (rotary_dim / (rotary_dim - 2)), which leaves
      the highest frequency and divides the lowest by factor;
    * ``"bands"``: with t = the turns a pair makes over the original context,
      frequencies of t > high_freq_factor are kept, of t < low_freq_factor
      divided by factor, and blended linearly in t between;
    * ``"yarn"``: the same with the blend linear in the pair's index between
      those that make beta_fast turns (kept) and beta_slow turns (divided); its
      amplitude is ``rope_amplitude(factor)``.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not base > 1.0 or not math.isfinite(base):
        raise ValueError("base must be finite and above 1")
    if not factor > 0.0 or not math.isfinite(factor):
        raise ValueError("factor must be positive and finite")
    i = np.arange(0, rotary_dim, 2, dtype=np.float64)
    if scaling == "ntk":
        if rotary_dim <= 2:
            raise ValueError("ntk scaling needs rotary_dim > 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-i / rotary_dim)
    if scaling in ("bands", "yarn"):
        if original_max_position <= 0:
            raise ValueError(f"{scaling} scaling needs original_max_position")
        if scaling == "bands":
            if not high_freq_factor > low_freq_factor:
                raise ValueError("high_freq_factor must exceed low_freq_factor")
            turns = original_max_position * f / (2 * math.pi)
            keep = (turns - low_freq_factor) / (high_freq_factor - low_freq_factor)
        else:
            if not beta_fast > beta_slow > 0:
                raise ValueError("beta_fast must exceed beta_slow, both positive")

            def pair_of(turns):  # index (not whole) of the pair that makes so many turns
                return rotary_dim * math.log(original_max_position / (turns * 2 * math.pi)) / (2 * math.log(base))
            low = max(math.floor(pair_of(beta_fast)), 0)
            high = min(math.ceil(pair_of(beta_slow)), rotary_dim - 1)
            keep = 1.0 - (i / 2 - low) / max(high - low, 1e-3)
        keep = np.clip(keep, 0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling == "linear":
        f = f / factor
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.from_numpy(np.ascontiguousarray(f)).to(device)


def rope_amplitude(factor: float) -> float:
    """The amplitude of "yarn"-scaled rotations: 0.1 ln(factor) + 1 (1 for
    factor <= 1)."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0


def _device_of(*tensors: torch.Tensor) -> int:
    """The CUDA device index all the tensors share (None entries are skipped)."""
    dev = -1
    for t in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (no CPU path)")
        i = t.get_device()
        if dev < 0:
            dev = i
        elif i != dev:
            raise ValueError("all tensors must be on the same device")
    return dev


def _on(dev: int, fn, *args):
    """fn(*args) with device dev current."""
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return fn(*args)
    return fn(*args)


def _call(fn, dev: int, *args) -> None:
    """fn(*args, the current stream of device dev) with dev current."""
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _call(fn, dev, *args)
    status = fn(*args, _raw_stream(dev) if _raw_stream else _stream(torch.device("cuda", dev)))
    if status != PKV_OK:
        _check(status)


def _rope_args(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, interleaved, amplitude, q_out, dev):
    """Checks paged_kv_write_rope's tensors; returns (its C arguments up to
    the dtype, q_out)."""
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() or \
            not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, num_kv_heads, head_dim]")
    NB, bs, Hkv, D = k_cache.shape
    dtype, shape, qs, ks, vs = q.dtype, q.shape, q.stride(), k.stride(), v.stride()
    if dtype not in DTYPE or k.dtype != dtype or v.dtype != dtype:
        raise ValueError("q, k and v must share dtype bfloat16 or float32")
    T = shape[0] if len(shape) == 3 else -1
    if T < 0 or shape[2] != D or qs[2] != 1 or qs[1] != D:
        raise ValueError(f"q must be [T, Hq, {D}] with contiguous heads")
    rows = (T, Hkv, D)
    if k.shape != rows or v.shape != rows or ks[2] != 1 or ks[1] != D or vs[2] != 1 or vs[1] != D:
        raise ValueError(f"k and v must be [{T}, {Hkv}, {D}] with contiguous heads")
    if T > 1 and 0 in (qs[0], ks[0], vs[0]):  # the C call takes a stride of 0 for dense
        raise ValueError("q, k and v must not repeat one token's row (a token stride of 0)")
    if positions.shape != (T,) or positions.dtype != torch.int64 or not positions.is_contiguous():
        raise ValueError("positions must be contiguous int64 [T]")
    if slot_mapping.shape != (T,) or slot_mapping.dtype != torch.int64 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous int64 [T]")
    if inv_freq.dim() != 1 or inv_freq.dtype != torch.float64 or not inv_freq.is_contiguous() or \
            not 0 < 2 * inv_freq.shape[0] <= D:
        raise ValueError("inv_freq must be contiguous float64 [rotary_dim / 2] with rotary_dim <= head_dim")
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=q.device)
    elif q_out.shape != shape or q_out.dtype != dtype or not q_out.is_contiguous() or q_out.get_device() != dev:
        raise ValueError("q_out must be contiguous and match q")
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(),
            slot_mapping.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), T, NB, bs, shape[1],
            Hkv, D, 2 * inv_freq.shape[0], 1 if interleaved else 0, amplitude, qs[0] if T > 1 else 0,
            ks[0] if T > 1 else 0, vs[0] if T > 1 else 0, DTYPE[dtype])
    return args, q_out


def paged_kv_write_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                        inv_freq: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, *, interleaved: bool = False, amplitude: float = 1.0,
                        q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate a step's ``q [T, Hq, D]`` and ``k [T, Hkv, D]`` to ``positions
    [T]`` (int64) and scatter ``k`` and ``v`` into the pools at
    ``slot_mapping`` (< 0 skips), in one pass; returns the rotated q.

    ``inv_freq`` (float64 ``[rotary_dim / 2]``, see ``rope_frequencies``) sets
    how much of a head is rotated: elements from rotary_dim on are copied.
    Pairs are (i, i + rotary_dim / 2), or (2i, 2i + 1) with ``interleaved``.
    q, k and v may be views with a token stride (a fused projection);
    ``q_out`` may be ``q`` itself when q is contiguous."""
    dev = _device_of(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache)
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise ValueError("q, k, v, k_cache, v_cache must share dtype bfloat16 or float32")
    args, q_out = _rope_args(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, interleaved, amplitude,
                             q_out, dev)
    _call(lib().paged_kv_write_rope, dev, *args)
    return q_out


def paged_kv_write_rope_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                            inv_freq: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, k_scale: float, v_scale: float, *, interleaved: bool = False,
                            amplitude: float = 1.0, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """``paged_kv_write_rope`` into FP8 pools: the codes are those of the
    rotated fp32 values, encoded as ``paged_kv_write_fp8`` does."""
    dev = _device_of(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache)
    _check_fp8_pools(k_cache, v_cache)
    args, q_out = _rope_args(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, interleaved, amplitude,
                             q_out, dev)
    _call(lib().paged_kv_write_rope_fp8, dev, *args, k_scale, v_scale)
    return q_out


# ----------------------------------------------------------------------------
# keeping the cache within a budget (include/paged_kv_budget.h)
# ----------------------------------------------------------------------------

def scores_workspace_size(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                          max_context: int) -> int:
    return int(lib().paged_attention_scores_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                                           max_context))


def scores_workspace_min(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                         max_context: int) -> int:
    return int(lib().paged_attention_scores_workspace_min(num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                                          max_context))


def _check_scores(scores, Hkv, score_rows, B) -> tuple:
    """Checks the running scores and their rows; returns scores' shape."""
    shape = scores.shape
    if scores.dtype != torch.float32 or len(shape) != 3 or (Hkv is not None and shape[1] != Hkv) or \
            not scores.is_contiguous():
        raise ValueError("scores must be contiguous float32 [num_rows, num_kv_heads, max_len]")
    if score_rows is not None:
        if score_rows.dtype != torch.int32 or score_rows.shape != (B,) or not score_rows.is_contiguous():
            raise ValueError("score_rows must be contiguous int32 [num_seqs]")
    elif shape[0] < B:
        raise ValueError("scores has fewer rows than the batch has sequences (pass score_rows)")
    return shape


def _scores_args(q, k_cache, block_tables, context_lens, query_start_loc, scores, scale, causal, decay, score_rows,
                 out, workspace, max_query_len, dev):
    """Checks paged_attention_scores' tensors; returns (its C arguments up to
    the decay, the workspace, out)."""
    qs, pool, table = q.shape, k_cache.shape, block_tables.shape
    if len(qs) != 3 or not q.is_contiguous():
        raise ValueError("q must be contiguous [T, Hq, D]")
    if len(pool) != 4 or not k_cache.is_contiguous():
        raise ValueError("the cache must be contiguous [num_blocks, block_size, num_kv_heads, head_dim]")
    T, Hq, D = qs
    NB, bs, Hkv, Dk = pool
    if Dk != D:
        raise ValueError("head_dim of q and the cache differ")
    if context_lens.dtype != torch.int32 or context_lens.dim() != 1 or not context_lens.is_contiguous():
        raise ValueError("context_lens must be contiguous int32 [num_seqs]")
    B = context_lens.shape[0]
    if block_tables.dtype != torch.int32 or len(table) != 2 or table[0] != B or (B > 0 and table[1] == 0) or \
            not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous int32 [num_seqs, max_blocks_per_seq], max_blocks_per_seq > 0")
    if query_start_loc.dtype != torch.int32 or query_start_loc.shape != (B + 1,) or \
            not query_start_loc.is_contiguous():
        raise ValueError(f"query_start_loc must be contiguous int32 [{B + 1}]")
    rows, _, length = _check_scores(scores, Hkv, score_rows, B)
    if out is None:
        out = scores
    elif out.shape != scores.shape or out.dtype != scores.dtype or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out must be contiguous and match scores")
    width = max(1, table[1])
    context = min(length, width * bs)
    if workspace is None:
        workspace = _on(dev, _workspace, q.device, scores_workspace_size(B, T, Hq, Hkv, context))
    elif workspace.dtype != torch.uint8 or workspace.get_device() != dev or \
            workspace.numel() < scores_workspace_min(B, T, Hq, Hkv, context):
        raise ValueError("workspace must be a uint8 CUDA tensor of at least scores_workspace_min bytes")
    args = (q.data_ptr(), k_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            query_start_loc.data_ptr(), None if score_rows is None else score_rows.data_ptr(), scores.data_ptr(),
            out.data_ptr(), B, T, Hq, Hkv, D, NB, bs, width, rows, length, int(max_query_len),
            scale, 1 if causal else 0, decay)
    return args, workspace, out


def paged_attention_scores(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, query_start_loc: torch.Tensor, scores: torch.Tensor,
                           scale: float, causal: bool = True, *, decay: float = 1.0,
                           score_rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, max_query_len: int = 0) -> torch.Tensor:
    """Add the attention weight that ``q [T, Hq, D]`` pays to each cached
    token to the running ``scores`` (float32 ``[num_rows, Hkv, max_len]``).

    ``scores[row, h, j]`` becomes ``decay`` times itself plus the softmax
    weights of cache position j, summed over the sequence's queries and the q
    heads of kv head h; at the positions of the step's own tokens (the last
    ones) it becomes that sum alone.  ``score_rows`` (int32 ``[num_seqs]``)
    names each sequence's row (default: its place in the batch; < 0 leaves it
    out).  The result goes to ``out`` (default: ``scores``, in place); entries
    past a sequence's length are left as they were.  ``max_query_len`` > 0
    promises that no sequence has more queries (a sequence that does is flagged
    and left out).  The other arguments are ``paged_attention_forward``'s;
    ``workspace`` (uint8, >= ``scores_workspace_min``) defaults to the cached
    buffer per (thread, device, stream)."""
    dev = _device_of(q, k_cache, block_tables, context_lens, query_start_loc, scores, score_rows)
    if q.dtype not in DTYPE or k_cache.dtype != q.dtype:
        raise ValueError("q and k_cache must share dtype bfloat16 or float32")
    args, ws, out = _scores_args(q, k_cache, block_tables, context_lens, query_start_loc, scores, scale, causal, decay,
                                 score_rows, out, workspace, max_query_len, dev)
    _call(lib().paged_attention_scores, dev, *args, ws.data_ptr(), ws.numel(), DTYPE[q.dtype])
    return out


def paged_attention_scores_fp8kv(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
                                 context_lens: torch.Tensor, query_start_loc: torch.Tensor, scores: torch.Tensor,
                                 scale: float, k_scale: float, causal: bool = True, *, decay: float = 1.0,
                                 score_rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                 workspace: torch.Tensor | None = None, max_query_len: int = 0) -> torch.Tensor:
    """``paged_attention_scores`` over an FP8 K pool read as code * k_scale
    (q bf16 with |q| below 65504, head_dim 128)."""
    dev = _device_of(q, k_cache, block_tables, context_lens, query_start_loc, scores, score_rows)
    _check_fp8_pools(k_cache, k_cache)
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16 with an FP8 cache")
    args, ws, out = _scores_args(q, k_cache, block_tables, context_lens, query_start_loc, scores, scale, causal, decay,
                                 score_rows, out, workspace, max_query_len, dev)
    _call(lib().paged_attention_scores_fp8kv, dev, *args, k_scale, ws.data_ptr(), ws.numel())
    return out


def paged_kv_select(scores: torch.Tensor, context_lens: torch.Tensor, budget: int, *, num_sink: int = 0,
                    num_recent: int = 0, score_rows: torch.Tensor | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """The positions ``budget`` keeps of each (sequence, kv head): int32
    ``[num_seqs, Hkv, budget]``, ascending, then -1.

    All of a sequence's L positions when L <= budget; else the first
    ``num_sink``, the last ``num_recent`` and the highest-scored between (ties
    to the lowest position)."""
    dev = _device_of(scores, context_lens, score_rows)
    if context_lens.dtype != torch.int32 or context_lens.dim() != 1 or not context_lens.is_contiguous():
        raise ValueError("context_lens must be contiguous int32 [num_seqs]")
    B = context_lens.shape[0]
    rows, Hkv, length = _check_scores(scores, None, score_rows, B)
    budget = int(budget)
    if out is None:
        out = torch.empty((B, Hkv, max(budget, 0)), dtype=torch.int32, device=scores.device)
    elif out.shape != (B, Hkv, budget) or out.dtype != torch.int32 or not out.is_contiguous() or \
            out.get_device() != dev:
        raise ValueError(f"out must be contiguous int32 {[B, Hkv, budget]}")
    _call(lib().paged_kv_select, dev, scores.data_ptr(), None if score_rows is None else score_rows.data_ptr(),
          context_lens.data_ptr(), out.data_ptr(), B, Hkv, rows, length, budget, int(num_sink), int(num_recent))
    return out


_POOL_DTYPE = dict(DTYPE)
_POOL_DTYPE.update({t: 2 for t in _FP8_TYPES})


def paged_kv_compact(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor, kept: torch.Tensor, *,
                     dst_block_tables: torch.Tensor | None = None, scores: torch.Tensor | None = None,
                     score_rows: torch.Tensor | None = None) -> None:
    """Move the kept tokens of each (sequence, kv head) to the front of its
    cache: position r becomes what position ``kept[s, h, r]`` was, in K, V
    and, if given, the running ``scores``.

    ``kept`` is ``paged_kv_select``'s int32 ``[num_seqs, Hkv, budget]``.  The
    rows go to ``dst_block_tables`` (default: in place): each of its blocks is
    the same entry of ``block_tables`` or a block no sequence of the call
    reads, as ``BlockManager.compact`` returns.  Pools are bf16, f32 or FP8."""
    dev = _device_of(k_cache, v_cache, block_tables, kept, dst_block_tables, scores, score_rows)
    pool, table, dtype = k_cache.shape, block_tables.shape, k_cache.dtype
    if dtype not in _POOL_DTYPE or v_cache.dtype != dtype:
        raise ValueError("k_cache and v_cache must share dtype bfloat16, float32 or FP8 (uint8, float8_e4m3fn)")
    if len(pool) != 4 or v_cache.shape != pool or not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, num_kv_heads, head_dim]")
    NB, bs, Hkv, D = pool
    if kept.dtype != torch.int32 or kept.dim() != 3 or kept.shape[1] != Hkv or not kept.is_contiguous():
        raise ValueError(f"kept must be contiguous int32 [num_seqs, {Hkv}, budget]")
    B, _, budget = kept.shape
    if block_tables.dtype != torch.int32 or len(table) != 2 or table[0] != B or (B > 0 and table[1] == 0) or \
            not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous int32 [num_seqs, max_blocks_per_seq], max_blocks_per_seq > 0")
    if dst_block_tables is not None and (dst_block_tables.dtype != torch.int32 or dst_block_tables.shape != table or
                                         not dst_block_tables.is_contiguous()):
        raise ValueError("dst_block_tables must be contiguous int32 of block_tables' shape")
    rows = length = 0
    if scores is not None:
        rows, _, length = _check_scores(scores, Hkv, score_rows, B)
    _call(lib().paged_kv_compact, dev, k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
          None if dst_block_tables is None else dst_block_tables.data_ptr(), kept.data_ptr(),
          None if score_rows is None else score_rows.data_ptr(), None if scores is None else scores.data_ptr(), B, Hkv,
          D, NB, bs, max(1, table[1]), budget, rows, length, _POOL_DTYPE[dtype])
