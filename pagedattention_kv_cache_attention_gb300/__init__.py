"""PagedAttention decode for GB300 (sm_103a): Python binding of libpa.

The functions here carry the names of the C ABI in ``include/pa.h`` and do
argument marshalling only: they check tensor devices, dtypes, shapes and
contiguity, pass ``data_ptr()`` values, sizes and the current CUDA stream to
the library, and turn a non-zero status into an exception.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback path, and
importing a function fails loudly when ``libpa.so`` has not been built.  (The
calls of rotated append and sparse attention make their checks in C++,
``csrc/pa_bind.cpp``.)

PyTorch supplies device memory and streams only.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "pa_reshape_and_cache", "pa_decode", "pa_decode_reduce", "pa_decode_workspace_size",
    "pa_decode_num_partitions", "pa_device_errors", "pa_status_string", "library_path",
    "pa_decode_static_workspace", "STATIC_WORKSPACE_BYTES", "pa_copy_blocks", "pa_swap_blocks",
    "pa_reshape_and_cache_fp8", "pa_decode_fp8", "pa_prefill", "pa_selftest_bounded_wait",
    "PaError", "DEVERR_BAD_BLOCK", "DEVERR_BAD_SLOT", "DEVERR_BAD_LEN", "DEVERR_TIMEOUT",
    "DEVERR_WORKSPACE", "DEVERR_PREFIX", "DECODE_COUNTER_BYTES", "new_decode_workspace",
    "pa_decode_shared_prefix", "pa_decode_shared_prefix_fp8", "pa_prefill_fp8",
    "pa_copy_blocks_fp8", "new_fp4_cache", "fp4_block_size", "pa_reshape_and_cache_fp4",
    "pa_gather_cache_fp4", "pa_decode_fp4", "pa_prefill_fp4",
    "new_rope_table", "new_key_bounds", "DEVERR_BAD_POS",
    "pa_rope_and_cache", "pa_rope_and_cache_fp8", "pa_rope_and_cache_fp4",
    "pa_update_key_bounds", "pa_update_key_bounds_fp8", "pa_update_key_bounds_fp4",
    "pa_select_blocks", "pa_decode_sparse", "pa_decode_sparse_fp8", "pa_decode_sparse_fp4",
]

PA_FP16, PA_BF16 = 0, 1
DEVERR_BAD_BLOCK, DEVERR_BAD_SLOT, DEVERR_BAD_LEN, DEVERR_TIMEOUT = 1, 2, 4, 8
DEVERR_WORKSPACE = 16
DEVERR_PREFIX = 32
DEVERR_BAD_POS = 64
# Bytes of join counters at the start of a split-context workspace
# (PA_DECODE_COUNTER_BYTES in include/pa.h); they must be zero when a
# workspace is first used, and every pa_decode call leaves them zero.
DECODE_COUNTER_BYTES = 256 * 1024
_DT = {torch.float16: PA_FP16, torch.bfloat16: PA_BF16}

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


class PaError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call}: {pa_status_string(status)} (status {status})")
        self.status = status


def library_path() -> str:
    return _build.LIB


def _load() -> ctypes.CDLL:
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                raise ImportError(
                    f"libpa.so is not built ({_build.LIB} missing): run "
                    "`python -c 'import __graft_entry__ as g; g.build()'` first")
            L = ctypes.CDLL(_build.LIB)
            P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            L.pa_reshape_and_cache.argtypes = [P, P, i64, i64, P, P, P, i32, i32, i32, i32, i64,
                                               i32, P]
            L.pa_reshape_and_cache.restype = i32
            L.pa_decode_num_partitions.argtypes = [i32, i32]
            L.pa_decode_num_partitions.restype = i32
            L.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
            L.pa_decode_workspace_size.restype = sz
            L.pa_decode.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i64,
                                    ctypes.c_float, i32, i32, P, sz, i32, P]
            L.pa_decode.restype = i32
            L.pa_decode_reduce.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, P]
            L.pa_decode_reduce.restype = i32
            L.pa_device_errors.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
            L.pa_selftest_bounded_wait.argtypes = [P]
            L.pa_selftest_bounded_wait.restype = i32
            L.pa_device_errors.restype = i32
            L.pa_status_string.argtypes = [i32]
            L.pa_status_string.restype = ctypes.c_char_p
            L.pa_version.restype = i32
            _lib = L
    return _lib


def pa_status_string(status: int) -> str:
    return _load().pa_status_string(int(status)).decode()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(call: str, status: int) -> None:
    if status != 0:
        raise PaError(call, status)


def _cuda(name: str, t: torch.Tensor, dtype=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{t.get_device()}, but the calls run on the current "
                         f"device cuda:{torch.cuda.current_device()}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}: fp16 or bf16")
    return _DT[t.dtype]


def pa_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, slot_mapping: torch.Tensor, stream=None) -> None:
    """Write key/value [T, Hkv, d] rows into k_cache/v_cache [NB, Hkv, bs, d]
    at slot_mapping[t] (int64; negative = skip), in place."""
    for n, t in (("key", key), ("value", value), ("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, k_cache.dtype)
    _cuda("slot_mapping", slot_mapping, torch.int64)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and slot_mapping.is_contiguous()):
        raise ValueError("caches and slot_mapping must be contiguous")
    T, Hkv, d = key.shape
    NB, Hkv2, bs, d2 = k_cache.shape
    if (Hkv, d) != (Hkv2, d2) or value.shape != key.shape or v_cache.shape != k_cache.shape:
        raise ValueError("key/value/cache shapes disagree")
    if slot_mapping.numel() != T:
        raise ValueError("slot_mapping must have one entry per token")
    for n, t in (("key", key), ("value", value)):
        if t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{n}: heads must be contiguous inside a token row")
    _check("pa_reshape_and_cache", _load().pa_reshape_and_cache(
        key.data_ptr(), value.data_ptr(), key.stride(0), value.stride(0), k_cache.data_ptr(),
        v_cache.data_ptr(), slot_mapping.data_ptr(), T, Hkv, d, bs, NB, _dtype_code(k_cache),
        _stream(stream)))


def pa_decode_num_partitions(max_context_len: int, partition_size: int) -> int:
    return int(_load().pa_decode_num_partitions(max_context_len, partition_size))


def pa_decode_workspace_size(num_seqs: int, num_q_heads: int, head_dim: int,
                             max_context_len: int, partition_size: int) -> int:
    return int(_load().pa_decode_workspace_size(num_seqs, num_q_heads, head_dim, max_context_len,
                                                partition_size))


def new_decode_workspace(num_seqs: int, num_q_heads: int, head_dim: int, max_context_len: int,
                         partition_size: int, device=None) -> torch.Tensor:
    """A zero-filled workspace (CUDA uint8 tensor) of pa_decode_workspace_size
    bytes, at least one byte; its join counters start at zero as pa_decode
    requires, and every pa_decode call leaves them zero, so it can be reused
    for any later call it is large enough for."""
    need = pa_decode_workspace_size(num_seqs, num_q_heads, head_dim, max_context_len,
                                    partition_size)
    return torch.zeros(max(1, need), dtype=torch.uint8,
                       device=device if device is not None else torch.cuda.current_device())


def pa_decode(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
              scale: float, max_context_len: int, partition_size: int = 0,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Paged decode attention into ``out`` [B, Hq, d].  ``workspace`` (a CUDA
    uint8 tensor of at least pa_decode_workspace_size bytes whose first
    DECODE_COUNTER_BYTES were zero when it was first used, e.g. from
    new_decode_workspace) is allocated here, zero-filled, with torch when it
    is needed and not given."""
    dt = k_cache.dtype
    for n, t in (("out", out), ("query", query), ("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, dt)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _cuda("block_tables", block_tables, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    if not (block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("block_tables and context_lens must be contiguous")
    B, Hq, d = query.shape
    NB, Hkv, bs, d2 = k_cache.shape
    if out.shape != query.shape or v_cache.shape != k_cache.shape or d2 != d:
        raise ValueError("out/query/cache shapes disagree")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_tables must be [B, MB] and context_lens [B]")
    need = pa_decode_workspace_size(B, Hq, d, max_context_len, partition_size)
    ws_ptr, ws_bytes = 0, 0
    if need:
        if workspace is None:
            workspace = torch.zeros(need, dtype=torch.uint8, device=query.device)
        _cuda("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check("pa_decode", _load().pa_decode(
        out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), B, Hq, Hkv, d,
        bs, NB, float(scale), int(max_context_len), int(partition_size), ws_ptr or None,
        ws_bytes, _dtype_code(k_cache), _stream(stream)))
    return out


def _shared_prefix(name, out, query, k_cache, v_cache, block_tables, context_lens, group_start,
                   prefix_lens, max_group_size, scale, scales, max_context_len, partition_size,
                   workspace, stream):
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    fp8 = scales is not None
    f = _blocks_fn(name, [P, P, P, P, P, i32, P, P, P, i32, i32, i32, i32, i32, i32, i32, i64, f32]
                   + ([f32, f32] if fp8 else []) + [i32, i32, P, ctypes.c_size_t, i32, P])
    for n, t in (("out", out), ("query", query)):
        _cuda(n, t, query.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, torch.uint8 if fp8 else query.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for n, t in (("block_tables", block_tables), ("context_lens", context_lens),
                 ("group_start", group_start), ("prefix_lens", prefix_lens)):
        _cuda(n, t, torch.int32)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    B, Hq, d = query.shape
    NB, Hkv, bs, d2 = k_cache.shape
    if out.shape != query.shape or v_cache.shape != k_cache.shape or d2 != d:
        raise ValueError("out/query/cache shapes disagree")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_tables must be [B, MB] and context_lens [B]")
    if prefix_lens.numel() != B or group_start.dim() != 1 or group_start.numel() < 2:
        raise ValueError("prefix_lens must be [B] and group_start [num_groups + 1]")
    need = pa_decode_workspace_size(B, Hq, d, max_context_len, partition_size)
    ws_ptr, ws_bytes = 0, 0
    if need:
        if workspace is None:
            workspace = torch.zeros(need, dtype=torch.uint8, device=query.device)
        _cuda("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(name, f(
        out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(),
        group_start.data_ptr(), prefix_lens.data_ptr(), group_start.numel() - 1,
        int(max_group_size), B, Hq, Hkv, d, bs, NB, float(scale),
        *([float(scales[0]), float(scales[1])] if fp8 else []), int(max_context_len),
        int(partition_size), ws_ptr or None, ws_bytes, _dtype_code(query), _stream(stream)))
    return out


def pa_decode_shared_prefix(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, group_start: torch.Tensor,
                            prefix_lens: torch.Tensor, max_group_size: int, scale: float,
                            max_context_len: int, partition_size: int,
                            workspace: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """pa_decode over groups of sequences sharing a prefix in the same
    physical blocks: ``group_start`` (int32 [num_groups + 1], runs of
    consecutive sequences covering the batch) and ``prefix_lens`` (int32 [B],
    shared leading tokens of each sequence, equal within a group) on the
    device; ``max_group_size`` bounds the groups' sizes.  The shared prefix's
    K/V is read once per group.  ``workspace`` as for pa_decode."""
    return _shared_prefix("pa_decode_shared_prefix", out, query, k_cache, v_cache, block_tables,
                          context_lens, group_start, prefix_lens, max_group_size, scale, None,
                          max_context_len, partition_size, workspace, stream)


def pa_decode_shared_prefix_fp8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                                v_cache: torch.Tensor, block_tables: torch.Tensor,
                                context_lens: torch.Tensor, group_start: torch.Tensor,
                                prefix_lens: torch.Tensor, max_group_size: int, scale: float,
                                k_scale: float, v_scale: float, max_context_len: int,
                                partition_size: int, workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """pa_decode_shared_prefix over uint8 FP8 E4M3 caches (codes times
    k_scale / v_scale), fp16 or bf16 queries and output."""
    return _shared_prefix("pa_decode_shared_prefix_fp8", out, query, k_cache, v_cache,
                          block_tables, context_lens, group_start, prefix_lens, max_group_size,
                          scale, (k_scale, v_scale), max_context_len, partition_size, workspace,
                          stream)


def pa_decode_reduce(out: torch.Tensor, workspace: torch.Tensor, context_lens: torch.Tensor,
                     max_context_len: int, partition_size: int, stream=None) -> torch.Tensor:
    """Join split-context partials in ``workspace`` into ``out`` [B, Hq, d]."""
    _cuda("out", out)
    _cuda("workspace", workspace)
    _cuda("context_lens", context_lens, torch.int32)
    if not (out.is_contiguous() and workspace.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("out, workspace and context_lens must be contiguous")
    B, Hq, d = out.shape
    _check("pa_decode_reduce", _load().pa_decode_reduce(
        out.data_ptr(), workspace.data_ptr(), context_lens.data_ptr(), B, Hq, d,
        int(max_context_len), int(partition_size), _dtype_code(out), _stream(stream)))
    return out


# Size of the library's own scratch array used by pa_decode_static_workspace
# (PA_STATIC_WORKSPACE_BYTES in include/pa.h).
STATIC_WORKSPACE_BYTES = 64 * 1024 * 1024


def pa_decode_static_workspace(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                               v_cache: torch.Tensor, block_tables: torch.Tensor,
                               context_lens: torch.Tensor, scale: float, max_context_len: int,
                               partition_size: int = 0, stream=None) -> torch.Tensor:
    """pa_decode for callers that may not allocate device memory (a framework
    that has reserved nearly all device memory for its own KV pool, a plugin
    whose host runtime owns every allocation, a real-time enqueue path that
    cannot risk an allocation's device-wide synchronisation): the
    split-context partials and join counters go to a fixed 64 MiB array the
    library carries, so neither this binding nor the library allocates.
    Shapes needing more scratch than that raise PaError (unsupported shape).
    All calls on a device share the array; calls that overlap on the GPU race."""
    L = _load()
    if not getattr(L.pa_decode_static_workspace, "argtypes", None):
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.pa_decode_static_workspace.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32,
                                                 i64, ctypes.c_float, i32, i32, i32, P]
        L.pa_decode_static_workspace.restype = i32
    dt = k_cache.dtype
    for n, t in (("out", out), ("query", query), ("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, dt)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _cuda("block_tables", block_tables, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    B, Hq, d = query.shape
    NB, Hkv, bs, _ = k_cache.shape
    _check("pa_decode_static_workspace", L.pa_decode_static_workspace(
        out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), B, Hq, Hkv, d,
        bs, NB, float(scale), int(max_context_len), int(partition_size), _dtype_code(k_cache),
        _stream(stream)))
    return out


def _blocks_fn(name: str, argtypes):
    L = _load()
    f = getattr(L, name)
    if not getattr(f, "argtypes", None):
        f.argtypes = argtypes
        f.restype = ctypes.c_int32
    return f


def _copy_blocks(name, k_cache, v_cache, block_mapping, dtypes, stream):
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    f = _blocks_fn(name, [P, P, P, i32, i32, i32, i32, i64, P])
    if k_cache.dtype not in dtypes:
        raise ValueError(f"{name}: caches must be {' or '.join(str(d) for d in dtypes)}")
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, k_cache.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _cuda("block_mapping", block_mapping, torch.int64)
    if block_mapping.dim() != 2 or block_mapping.shape[1] != 2 or not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be a contiguous [n, 2] tensor")
    NB, Hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    _check(name, f(k_cache.data_ptr(), v_cache.data_ptr(), block_mapping.data_ptr(),
                   block_mapping.shape[0], Hkv, d, bs, NB, _stream(stream)))


def pa_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, block_mapping: torch.Tensor,
                   stream=None) -> None:
    """Copy-on-write fork: for each row (src, dst) of ``block_mapping`` (CUDA
    int64 [n, 2]), physical block dst of both caches (fp16 or bf16) becomes a
    copy of block src.  Destinations distinct and not also sources."""
    _copy_blocks("pa_copy_blocks", k_cache, v_cache, block_mapping,
                 (torch.float16, torch.bfloat16), stream)


def pa_copy_blocks_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, block_mapping: torch.Tensor,
                       stream=None) -> None:
    """pa_copy_blocks over uint8 FP8 E4M3 caches."""
    _copy_blocks("pa_copy_blocks_fp8", k_cache, v_cache, block_mapping, (torch.uint8,), stream)


def pa_swap_blocks(src: torch.Tensor, dst: torch.Tensor, block_mapping: torch.Tensor,
                   stream=None) -> None:
    """Move whole blocks between pools [NB, ...] (one cache): dst block
    mapping[k, 1] = src block mapping[k, 0].  Each of src, dst is a CUDA tensor
    or a pinned CPU tensor; ``block_mapping`` is int64 [n, 2] on the GPU or in
    pinned CPU memory.  The copy runs as one kernel on ``stream``."""
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    f = _blocks_fn("pa_swap_blocks", [P, P, P, i32, i64, i64, i64, P])
    for n, t in (("src", src), ("dst", dst), ("block_mapping", block_mapping)):
        if not isinstance(t, torch.Tensor) or not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{n} must be a CUDA tensor or a pinned CPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if block_mapping.dtype != torch.int64 or block_mapping.dim() != 2 or block_mapping.shape[1] != 2:
        raise ValueError("block_mapping must be int64 [n, 2]")
    if src.dtype != dst.dtype or src.shape[1:] != dst.shape[1:]:
        raise ValueError("src and dst must have the same dtype and block shape")
    block_bytes = src[0].numel() * src.element_size() if src.shape[0] else 0
    _check("pa_swap_blocks", f(src.data_ptr(), dst.data_ptr(), block_mapping.data_ptr(),
                               block_mapping.shape[0], block_bytes, src.shape[0], dst.shape[0],
                               _stream(stream)))


def pa_reshape_and_cache_fp8(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, slot_mapping: torch.Tensor, k_scale: float,
                             v_scale: float, stream=None) -> None:
    """Write key/value [T, Hkv, d] (fp16/bf16) into uint8 FP8 E4M3 caches
    [NB, Hkv, bs, d] at slot_mapping[t], each element as the code of x/scale."""
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    f = _blocks_fn("pa_reshape_and_cache_fp8", [P, P, i64, i64, P, P, P, i32, i32, i32, i32,
                                                 i64, i32, f32, f32, P])
    for n, t in (("key", key), ("value", value)):
        _cuda(n, t, key.dtype)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n}: heads must be contiguous inside a token row")
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, torch.uint8)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _cuda("slot_mapping", slot_mapping, torch.int64)
    T, Hkv, d = key.shape
    NB, Hkv2, bs, d2 = k_cache.shape
    if (Hkv, d) != (Hkv2, d2) or value.shape != key.shape or v_cache.shape != k_cache.shape:
        raise ValueError("key/value/cache shapes disagree")
    _check("pa_reshape_and_cache_fp8", f(
        key.data_ptr(), value.data_ptr(), key.stride(0), value.stride(0), k_cache.data_ptr(),
        v_cache.data_ptr(), slot_mapping.data_ptr(), T, Hkv, d, bs, NB, _dtype_code(key),
        float(k_scale), float(v_scale), _stream(stream)))


def pa_decode_fp8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                  scale: float, k_scale: float, v_scale: float, max_context_len: int,
                  partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Paged decode attention over uint8 FP8 E4M3 caches (codes times
    k_scale / v_scale) into ``out`` [B, Hq, d] (fp16 or bf16 queries and output)."""
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    f = _blocks_fn("pa_decode_fp8", [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i64, f32,
                                     f32, f32, i32, i32, P, sz, i32, P])
    for n, t in (("out", out), ("query", query)):
        _cuda(n, t, query.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, torch.uint8)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _cuda("block_tables", block_tables, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    B, Hq, d = query.shape
    NB, Hkv, bs, _ = k_cache.shape
    need = pa_decode_workspace_size(B, Hq, d, max_context_len, partition_size)
    ws_ptr, ws_bytes = 0, 0
    if need:
        if workspace is None:
            workspace = torch.zeros(need, dtype=torch.uint8, device=query.device)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check("pa_decode_fp8", f(
        out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), B, Hq, Hkv, d,
        bs, NB, float(scale), float(k_scale), float(v_scale), int(max_context_len),
        int(partition_size), ws_ptr or None, ws_bytes, _dtype_code(query), _stream(stream)))
    return out


def _prefill(name, out, query, query_start, k_cache, v_cache, block_tables, context_lens, scale,
             scales, max_q_len, stream):
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    fp8 = scales is not None
    f = _blocks_fn(name, [P, P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i64, f32]
                   + ([f32, f32] if fp8 else []) + [i32, P])
    for n, t in (("out", out), ("query", query)):
        _cuda(n, t, query.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _cuda(n, t, torch.uint8 if fp8 else query.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for n, t in (("query_start", query_start), ("block_tables", block_tables),
                 ("context_lens", context_lens)):
        _cuda(n, t, torch.int32)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    total_q, Hq, d = query.shape
    NB, Hkv, bs, _ = k_cache.shape
    B = context_lens.numel()
    if query_start.numel() != B + 1 or out.shape != query.shape:
        raise ValueError("query_start must have num_seqs + 1 entries; out must match query")
    _check(name, f(out.data_ptr(), query.data_ptr(), query_start.data_ptr(), k_cache.data_ptr(),
                   v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
                   context_lens.data_ptr(), B, int(max_q_len), Hq, Hkv, d, bs, NB, float(scale),
                   *([float(scales[0]), float(scales[1])] if fp8 else []), _dtype_code(query),
                   _stream(stream)))
    return out


def pa_prefill(out: torch.Tensor, query: torch.Tensor, query_start: torch.Tensor,
               k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, scale: float, max_q_len: int,
               stream=None) -> torch.Tensor:
    """Causal chunked-prefill attention into ``out`` [total_q, Hq, d]: row t of
    sequence i's chunk (rows query_start[i]..query_start[i+1]-1) sits at
    position context_lens[i] - q_len_i + t and attends to tokens 0..that."""
    return _prefill("pa_prefill", out, query, query_start, k_cache, v_cache, block_tables,
                    context_lens, scale, None, max_q_len, stream)


def pa_prefill_fp8(out: torch.Tensor, query: torch.Tensor, query_start: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                   context_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float,
                   max_q_len: int, stream=None) -> torch.Tensor:
    """pa_prefill over uint8 FP8 E4M3 caches (codes times k_scale / v_scale),
    fp16 or bf16 queries and output."""
    return _prefill("pa_prefill_fp8", out, query, query_start, k_cache, v_cache, block_tables,
                    context_lens, scale, (k_scale, v_scale), max_q_len, stream)


def new_fp4_cache(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int,
                  device=None) -> torch.Tensor:
    """A zero-filled FP4 cache (K or V): uint8 [num_blocks, num_kv_heads,
    block_size * head_dim * 9 / 16], each (block, head) holding its tokens'
    E2M1 codes [block_size, head_dim / 2] (the even element of a byte in the
    low nibble) and then their E4M3 scales [block_size, head_dim / 16]."""
    return torch.zeros(num_blocks, num_kv_heads, block_size * head_dim * 9 // 16,
                       dtype=torch.uint8,
                       device=device if device is not None else torch.cuda.current_device())


def fp4_block_size(cache: torch.Tensor, head_dim: int) -> int:
    """Tokens per block of an FP4 cache for heads of ``head_dim``."""
    if cache.dim() != 3 or cache.shape[2] * 16 % (9 * head_dim):
        raise ValueError(f"an FP4 cache is uint8 [NB, Hkv, block_size * d * 9 / 16]; "
                         f"{tuple(cache.shape)} is none for d = {head_dim}")
    return cache.shape[2] * 16 // (9 * head_dim)


# The FP4 calls check their arguments in one pass and look nothing up twice: for
# a decode step of a few short sequences the host's share of a call is longer
# than the kernel (16 us a call with the checks of the calls above, 8 with these).
# What fits passes one expression; only what does not is gone through tensor by
# tensor, to name it.
_fp4_fns = {}
_U8, _I32, _I64 = torch.uint8, torch.int32, torch.int64
_FP4_ARGS = {
    "cache": "PPllPPPiiiiliffP",                  # write and read-back
    "decode": "PPPPPiPiiiiilfffiiPziP",
    "prefill": "PPPPPPiPiiiiiilfffiP",
}
_CT = {"P": ctypes.c_void_p, "i": ctypes.c_int32, "l": ctypes.c_int64, "f": ctypes.c_float,
       "z": ctypes.c_size_t}


def _fp4_fn(name: str, kind: str):
    f = getattr(_load(), name)
    f.argtypes, f.restype = [_CT[c] for c in _FP4_ARGS[kind]], ctypes.c_int32
    _fp4_fns[name] = f
    return f


def _fits(name: str, t, dtype, dev: int) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.is_contiguous()):
        return
    _cuda(name, t, dtype)
    raise ValueError(f"{name} must be contiguous")


# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


# (asked only where a CUDA tensor is at hand, so CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(name: str, t) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = _current_device()
    if t.get_device() != dev:
        _cuda(name, t)
    return dev


def _all_fit(dev: int, **tensors) -> None:
    """Each name=(tensor, dtype): dense on the current device; raises for the first that is not."""
    for name, (t, dtype) in tensors.items():
        _fits(name, t, dtype, dev)


def _cache_fp4(name, key, value, k_cache, v_cache, slot_mapping, k_scale, v_scale, stream):
    f = _fp4_fns.get(name) or _fp4_fn(name, "cache")
    dev = _device_of("key", key)
    shape, dtype = key.shape, key.dtype
    if len(shape) != 3 or not isinstance(value, torch.Tensor) or value.shape != shape:
        raise ValueError("key and value must be [T, Hkv, d], alike")
    T, Hkv, d = shape
    if not value.is_cuda or value.get_device() != dev or value.dtype is not dtype:
        _cuda("value", value, dtype)
    ks, vs = key.stride(), value.stride()
    if ks[2] != 1 or ks[1] != d or vs[2] != 1 or vs[1] != d:
        raise ValueError("key, value: heads must be contiguous inside a token row")
    try:
        fit = (k_cache.dtype is _U8 and v_cache.dtype is _U8 and slot_mapping.dtype is _I64
               and k_cache.get_device() == dev == v_cache.get_device() == slot_mapping.get_device()
               and k_cache.is_contiguous() and v_cache.is_contiguous()
               and slot_mapping.is_contiguous())
    except AttributeError:
        fit = False
    if not fit:
        _all_fit(dev, k_cache=(k_cache, _U8), v_cache=(v_cache, _U8),
                 slot_mapping=(slot_mapping, _I64))
    cache = k_cache.shape
    if v_cache.shape != cache:
        raise ValueError("k_cache and v_cache shapes differ")
    bs = fp4_block_size(k_cache, d)
    if cache[1] != Hkv:
        raise ValueError("key/value/cache shapes disagree")
    if slot_mapping.numel() != T:
        raise ValueError("slot_mapping must have one entry per token")
    row = Hkv * d  # the stride of a single row is not looked at
    st = f(key.data_ptr(), value.data_ptr(), ks[0] if T > 1 else row, vs[0] if T > 1 else row,
           k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), T, Hkv, d, bs,
           cache[0], _dtype_code(key), float(k_scale), float(v_scale),
           _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise PaError(name, st)


def pa_reshape_and_cache_fp4(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                             k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Write key/value [T, Hkv, d] (fp16/bf16) into FP4 caches (new_fp4_cache)
    at slot_mapping[t] (int64; negative = skip), quantised in groups of 16."""
    _cache_fp4("pa_reshape_and_cache_fp4", key, value, k_cache, v_cache, slot_mapping, k_scale,
               v_scale, stream)


def pa_gather_cache_fp4(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, slot_mapping: torch.Tensor, k_scale: float = 1.0,
                        v_scale: float = 1.0, stream=None) -> None:
    """Read cached tokens back: row t of ``key`` and ``value`` (fp16/bf16 [T,
    Hkv, d], written in place) becomes the values cached at slot_mapping[t]
    (int64; a negative slot leaves its row as it was)."""
    _cache_fp4("pa_gather_cache_fp4", key, value, k_cache, v_cache, slot_mapping, k_scale,
               v_scale, stream)


def pa_decode_fp4(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                  scale: float, k_scale: float, v_scale: float, max_context_len: int,
                  partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Paged decode attention over FP4 caches into ``out`` [B, Hq, d] (fp16 or
    bf16 queries and output).  ``workspace`` as for pa_decode."""
    f = _fp4_fns.get("pa_decode_fp4") or _fp4_fn("pa_decode_fp4", "decode")
    dev = _device_of("query", query)
    dtype = query.dtype
    try:
        fit = (out.dtype is dtype and k_cache.dtype is _U8 and v_cache.dtype is _U8
               and block_tables.dtype is _I32 and context_lens.dtype is _I32
               and out.get_device() == dev == k_cache.get_device() == v_cache.get_device()
               and block_tables.get_device() == dev == context_lens.get_device()
               and query.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous()
               and v_cache.is_contiguous() and block_tables.is_contiguous()
               and context_lens.is_contiguous())
    except AttributeError:
        fit = False
    if not fit:
        _all_fit(dev, query=(query, dtype), out=(out, dtype), k_cache=(k_cache, _U8),
                 v_cache=(v_cache, _U8), block_tables=(block_tables, _I32),
                 context_lens=(context_lens, _I32))
    shape, cache, table = query.shape, k_cache.shape, block_tables.shape
    B, Hq, d = shape
    if v_cache.shape != cache:
        raise ValueError("k_cache and v_cache shapes differ")
    bs = fp4_block_size(k_cache, d)
    if out.shape != shape:
        raise ValueError("out and query shapes differ")
    if len(table) != 2 or table[0] != B or context_lens.numel() != B:
        raise ValueError("block_tables must be [B, MB] and context_lens [B]")
    ws_ptr, ws_bytes = None, 0
    if 0 < partition_size < max_context_len:
        if workspace is None:
            # made on the call's own stream: its zeros come before the kernels, and its
            # memory is not handed on before they are done
            handle = _raw_stream(dev) if stream is None else _stream(stream)
            on = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
            with torch.cuda.stream(on):
                workspace = new_decode_workspace(B, Hq, d, max_context_len, partition_size, dev)
        _cuda("workspace", workspace)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = f(out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
           block_tables.data_ptr(), table[1], context_lens.data_ptr(), B, Hq,
           cache[1], d, bs, cache[0], float(scale), float(k_scale), float(v_scale),
           int(max_context_len), int(partition_size), ws_ptr, ws_bytes, _dtype_code(query),
           _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise PaError("pa_decode_fp4", st)
    return out


def pa_prefill_fp4(out: torch.Tensor, query: torch.Tensor, query_start: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                   context_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float,
                   max_q_len: int, stream=None) -> torch.Tensor:
    """pa_prefill over FP4 caches, fp16 or bf16 queries and output."""
    f = _fp4_fns.get("pa_prefill_fp4") or _fp4_fn("pa_prefill_fp4", "prefill")
    dev = _device_of("query", query)
    dtype = query.dtype
    try:
        fit = (out.dtype is dtype and k_cache.dtype is _U8 and v_cache.dtype is _U8
               and query_start.dtype is _I32 and block_tables.dtype is _I32
               and context_lens.dtype is _I32
               and out.get_device() == dev == k_cache.get_device() == v_cache.get_device()
               and query_start.get_device() == dev == block_tables.get_device()
               and context_lens.get_device() == dev
               and query.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous()
               and v_cache.is_contiguous() and query_start.is_contiguous()
               and block_tables.is_contiguous() and context_lens.is_contiguous())
    except AttributeError:
        fit = False
    if not fit:
        _all_fit(dev, query=(query, dtype), out=(out, dtype), k_cache=(k_cache, _U8),
                 v_cache=(v_cache, _U8), query_start=(query_start, _I32),
                 block_tables=(block_tables, _I32), context_lens=(context_lens, _I32))
    shape, cache, table = query.shape, k_cache.shape, block_tables.shape
    total_q, Hq, d = shape
    if v_cache.shape != cache:
        raise ValueError("k_cache and v_cache shapes differ")
    bs = fp4_block_size(k_cache, d)
    B = context_lens.numel()
    if query_start.numel() != B + 1 or out.shape != shape:
        raise ValueError("query_start must have num_seqs + 1 entries; out must match query")
    if len(table) != 2 or table[0] != B:
        raise ValueError("block_tables must be [B, MB]")
    st = f(out.data_ptr(), query.data_ptr(), query_start.data_ptr(), k_cache.data_ptr(),
           v_cache.data_ptr(), block_tables.data_ptr(), table[1],
           context_lens.data_ptr(), B, int(max_q_len), Hq, cache[1], d, bs,
           cache[0], float(scale), float(k_scale), float(v_scale), _dtype_code(query),
           _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise PaError("pa_prefill_fp4", st)
    return out


def new_rope_table(max_position: int, rotary_dim: int, base: float = 10000.0,
                   device=None) -> torch.Tensor:
    """The table that pa_rope_and_cache reads: fp32 [max_position, rotary_dim],
    cosines and then sines of position * base^(-2 i / rotary_dim), the angles
    formed in 64 bits.  (Any other table of that form does as well.)"""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    dev = device if device is not None else torch.cuda.current_device()
    freq = float(base) ** (-torch.arange(rotary_dim // 2, dtype=torch.float64, device=dev)
                           * 2 / rotary_dim)
    angle = torch.arange(max_position, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def new_key_bounds(num_blocks: int, num_kv_heads: int, head_dim: int, device=None):
    """(bounds, bound_scales) of zeros for the blocks of a pool: int8
    [num_blocks, num_kv_heads, 2, head_dim] and fp32 [num_blocks, num_kv_heads]."""
    dev = device if device is not None else torch.cuda.current_device()
    return (torch.zeros(num_blocks, num_kv_heads, 2, head_dim, dtype=torch.int8, device=dev),
            torch.zeros(num_blocks, num_kv_heads, dtype=torch.float32, device=dev))


# These calls go through pa_bind.cpp, which makes the checks below and the C call
# in C++; only what does not fit there is gone through here, to name it.
_bind = None


def _native():
    """The module built from pa_bind.cpp."""
    global _bind
    _load()
    if not os.path.exists(_build.BIND):
        raise ImportError(f"{_build.BIND} is missing (it belongs to one torch and one Python): run "
                          "`python -c 'import __graft_entry__ as g; g.build()'` first")
    spec = importlib.util.spec_from_file_location("pa_bind", _build.BIND)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.set_raw_stream(_raw_stream)
    _bind = module
    return module


_I8, _F32 = torch.int8, torch.float32
_SPARSE_ARGS = {
    "pa_rope_and_cache": "PPPPllllPPPPPiiiiiiilliP", "pa_update_key_bounds": "PPPPiPPiiiiiliP",
    "pa_select_blocks": "PPPPPPiPPiiiiiiliiiiiP", "pa_decode_sparse": "PPPPPPiiiiiilfiP",
    "pa_rope_and_cache_fp8": "PPPPllllPPPPPiiiiiiilliffP",
    "pa_rope_and_cache_fp4": "PPPPllllPPPPPiiiiiiilliffP",
    "pa_update_key_bounds_fp8": "PPPPiPPiiiiilP", "pa_update_key_bounds_fp4": "PPPPiPPiiiiilP",
    "pa_decode_sparse_fp8": "PPPPPPiiiiiilfffiP", "pa_decode_sparse_fp4": "PPPPPPiiiiiilfffiP",
}


def _sparse_fn(name: str):
    f = getattr(_load(), name)
    f.argtypes, f.restype = [_CT[c] for c in _SPARSE_ARGS[name]], ctypes.c_int32
    return f


def _cache_shape(name: str, cache: torch.Tensor, d: int):
    """(num_blocks, num_kv_heads, block_size) of a cache for heads of ``d``."""
    shape = cache.shape
    if name.endswith("_fp4"):
        return shape[0], shape[1], fp4_block_size(cache, d)
    if len(shape) != 4 or shape[3] != d:
        raise ValueError(f"a cache is [NB, Hkv, block_size, d = {d}], got {tuple(shape)}")
    return shape[0], shape[1], shape[2]


def _rope(name, query_out, query, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
          scales, interleaved, stream):
    dev = _device_of("query", query)
    dtype = query.dtype
    strides = []
    for n, t in (("query_out", query_out), ("query", query), ("key", key), ("value", value)):
        _cuda(n, t, dtype)
        if t.dim() != 3:
            raise ValueError(f"{n} must be [T, heads, d]")
        st, (rows, heads, d) = t.stride(), t.shape
        if (st[2] != 1 and d > 1) or (st[1] != d and heads > 1):
            raise ValueError(f"{n}: heads must be contiguous inside a token row")
        # (the stride of a single row is not looked at)
        strides.append(st[0] if rows > 1 else heads * d)
    cache = _U8 if scales else dtype
    _all_fit(dev, k_cache=(k_cache, cache), v_cache=(v_cache, cache),
             slot_mapping=(slot_mapping, _I64), positions=(positions, _I64),
             cos_sin=(cos_sin, _F32))
    T, Hq, d = query.shape
    Hkv = key.shape[1]
    if query_out.shape != query.shape:
        raise ValueError("query_out must match query")
    if key.shape != (T, Hkv, d) or value.shape != key.shape:
        raise ValueError("key and value must be [T, Hkv, d], with query's T and d")
    NB, heads, bs = _cache_shape(name, k_cache, d)
    if heads != Hkv or v_cache.shape != k_cache.shape:
        raise ValueError("key/value/cache shapes disagree")
    if slot_mapping.numel() != T or positions.numel() != T:
        raise ValueError("slot_mapping and positions must have one entry per token")
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_position, rotary_dim]")
    _check(name, _sparse_fn(name)(
        query_out.data_ptr(), query.data_ptr(), key.data_ptr(), value.data_ptr(), *strides,
        k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(),
        cos_sin.data_ptr(), T, Hq, Hkv, d, cos_sin.shape[1], 1 if interleaved else 0, bs, NB,
        cos_sin.shape[0], _dtype_code(query), *scales, _stream(stream)))
    return query_out


def pa_rope_and_cache(query_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                      value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                      interleaved: bool = False, stream=None) -> torch.Tensor:
    """Rotate query [T, Hq, d] and key [T, Hkv, d] by positions [T] (int64) with
    the table cos_sin (new_rope_table); write the queries into ``query_out``
    (which may be ``query``), and keys and values into the caches at
    slot_mapping[t] (int64; a token with a negative slot is left out)."""
    st = (_bind or _native()).rope(0, query_out, query, key, value, k_cache, v_cache,
                                   slot_mapping, positions, cos_sin, 1.0, 1.0, interleaved,
                                   stream)
    if st == 0:
        return query_out
    if st > 0:
        raise PaError("pa_rope_and_cache", st)
    return _rope("pa_rope_and_cache", query_out, query, key, value, k_cache, v_cache,
                 slot_mapping, positions, cos_sin, (), interleaved, stream)


def pa_rope_and_cache_fp8(query_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                          value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          slot_mapping: torch.Tensor, positions: torch.Tensor,
                          cos_sin: torch.Tensor, k_scale: float, v_scale: float,
                          interleaved: bool = False, stream=None) -> torch.Tensor:
    """pa_rope_and_cache into uint8 FP8 E4M3 caches."""
    st = (_bind or _native()).rope(1, query_out, query, key, value, k_cache, v_cache,
                                   slot_mapping, positions, cos_sin, k_scale, v_scale, interleaved,
                                   stream)
    if st == 0:
        return query_out
    if st > 0:
        raise PaError("pa_rope_and_cache_fp8", st)
    return _rope("pa_rope_and_cache_fp8", query_out, query, key, value, k_cache, v_cache,
                 slot_mapping, positions, cos_sin, (float(k_scale), float(v_scale)), interleaved,
                 stream)


def pa_rope_and_cache_fp4(query_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                          value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          slot_mapping: torch.Tensor, positions: torch.Tensor,
                          cos_sin: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0,
                          interleaved: bool = False, stream=None) -> torch.Tensor:
    """pa_rope_and_cache into FP4 caches (new_fp4_cache)."""
    st = (_bind or _native()).rope(2, query_out, query, key, value, k_cache, v_cache,
                                   slot_mapping, positions, cos_sin, k_scale, v_scale, interleaved,
                                   stream)
    if st == 0:
        return query_out
    if st > 0:
        raise PaError("pa_rope_and_cache_fp4", st)
    return _rope("pa_rope_and_cache_fp4", query_out, query, key, value, k_cache, v_cache,
                 slot_mapping, positions, cos_sin, (float(k_scale), float(v_scale)), interleaved,
                 stream)


def _key_bounds(name, bounds, bound_scales, k_cache, block_tables, context_lens, query_start,
                max_q_len, stream):
    dev = _device_of("k_cache", k_cache)
    plain = name == "pa_update_key_bounds"
    _all_fit(dev, bounds=(bounds, _I8), bound_scales=(bound_scales, _F32),
             k_cache=(k_cache, k_cache.dtype if plain else _U8),
             block_tables=(block_tables, _I32), context_lens=(context_lens, _I32))
    start = _start(query_start, dev, context_lens)
    shape = bounds.shape
    if len(shape) != 4 or shape[2] != 2 or bound_scales.shape != shape[:2]:
        raise ValueError("bounds must be [NB, Hkv, 2, d] and bound_scales [NB, Hkv]")
    d = shape[3]
    NB, Hkv, bs = _cache_shape(name, k_cache, d)
    if shape[0] != NB or shape[1] != Hkv:
        raise ValueError("bounds and k_cache differ in blocks or heads")
    B = context_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [B, MB] and context_lens [B]")
    _check(name, _sparse_fn(name)(
        bounds.data_ptr(), bound_scales.data_ptr(), k_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], context_lens.data_ptr(), start, B, int(max_q_len), Hkv, d, bs, NB,
        *((_dtype_code(k_cache),) if plain else ()), _stream(stream)))


def _start(query_start, dev, context_lens):
    """The address of query_start, checked; None for none."""
    if query_start is None:
        return None
    _fits("query_start", query_start, _I32, dev)
    if query_start.numel() != context_lens.numel() + 1:
        raise ValueError("query_start must have num_seqs + 1 entries")
    return query_start.data_ptr()


def pa_update_key_bounds(bounds: torch.Tensor, bound_scales: torch.Tensor, k_cache: torch.Tensor,
                         block_tables: torch.Tensor, context_lens: torch.Tensor,
                         query_start: Optional[torch.Tensor] = None, max_q_len: int = 1,
                         stream=None) -> None:
    """Bring ``bounds`` and ``bound_scales`` (new_key_bounds) up to date for the
    blocks that hold the newest tokens of each sequence: the last one, or the
    last query_start[i + 1] - query_start[i] (at most max_q_len)."""
    st = (_bind or _native()).key_bounds(0, bounds, bound_scales, k_cache, block_tables,
                                         context_lens, query_start, max_q_len, stream)
    if st == 0:
        return
    if st > 0:
        raise PaError("pa_update_key_bounds", st)
    _key_bounds("pa_update_key_bounds", bounds, bound_scales, k_cache, block_tables,
                context_lens, query_start, max_q_len, stream)


def pa_update_key_bounds_fp8(bounds: torch.Tensor, bound_scales: torch.Tensor,
                             k_cache: torch.Tensor, block_tables: torch.Tensor,
                             context_lens: torch.Tensor,
                             query_start: Optional[torch.Tensor] = None, max_q_len: int = 1,
                             stream=None) -> None:
    """pa_update_key_bounds over a uint8 FP8 E4M3 cache."""
    st = (_bind or _native()).key_bounds(1, bounds, bound_scales, k_cache, block_tables,
                                         context_lens, query_start, max_q_len, stream)
    if st == 0:
        return
    if st > 0:
        raise PaError("pa_update_key_bounds_fp8", st)
    _key_bounds("pa_update_key_bounds_fp8", bounds, bound_scales, k_cache, block_tables,
                context_lens, query_start, max_q_len, stream)


def pa_update_key_bounds_fp4(bounds: torch.Tensor, bound_scales: torch.Tensor,
                             k_cache: torch.Tensor, block_tables: torch.Tensor,
                             context_lens: torch.Tensor,
                             query_start: Optional[torch.Tensor] = None, max_q_len: int = 1,
                             stream=None) -> None:
    """pa_update_key_bounds over an FP4 cache."""
    st = (_bind or _native()).key_bounds(2, bounds, bound_scales, k_cache, block_tables,
                                         context_lens, query_start, max_q_len, stream)
    if st == 0:
        return
    if st > 0:
        raise PaError("pa_update_key_bounds_fp4", st)
    _key_bounds("pa_update_key_bounds_fp4", bounds, bound_scales, k_cache, block_tables,
                context_lens, query_start, max_q_len, stream)


def pa_select_blocks(selected_tables: torch.Tensor, selected_lens: torch.Tensor,
                     query: torch.Tensor, bounds: torch.Tensor, bound_scales: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor, block_size: int,
                     max_context_len: int, num_sink: int = 1, num_recent: int = 1,
                     query_start: Optional[torch.Tensor] = None, max_q_len: int = 1,
                     stream=None):
    """For every row of query [R, Hq, d] and KV head, pick the K blocks whose
    bounds promise the largest logits: their physical ids into
    ``selected_tables`` (int32 [R, Hkv, K], -1 behind them) and the tokens in
    them into ``selected_lens`` (int32 [R, Hkv]), for pa_decode_sparse.  Row i
    is sequence i's query, or rows query_start[i] .. query_start[i + 1] - 1 its
    last tokens.  The first num_sink and last num_recent blocks that a row
    sees are always taken.  Returns (selected_tables, selected_lens)."""
    st = (_bind or _native()).select(selected_tables, selected_lens, query, bounds, bound_scales,
                                     block_tables, context_lens, block_size, max_context_len,
                                     num_sink, num_recent, query_start, max_q_len, stream)
    if st == 0:
        return selected_tables, selected_lens
    if st > 0:
        raise PaError("pa_select_blocks", st)
    dev = _device_of("query", query)
    _all_fit(dev, query=(query, query.dtype), selected_tables=(selected_tables, _I32),
             selected_lens=(selected_lens, _I32), bounds=(bounds, _I8),
             bound_scales=(bound_scales, _F32), block_tables=(block_tables, _I32),
             context_lens=(context_lens, _I32))
    start = _start(query_start, dev, context_lens)
    shape, picked = bounds.shape, selected_tables.shape
    if query.dim() != 3 or len(picked) != 3:
        raise ValueError("query must be [R, Hq, d] and selected_tables [R, Hkv, K]")
    R, Hq, d = query.shape
    if len(shape) != 4 or shape[2] != 2 or shape[3] != d or bound_scales.shape != shape[:2]:
        raise ValueError("bounds must be [NB, Hkv, 2, d] and bound_scales [NB, Hkv]")
    NB, Hkv = shape[:2]
    if picked[:2] != (R, Hkv) or selected_lens.shape != picked[:2]:
        raise ValueError("selected_tables must be [R, Hkv, K] and selected_lens [R, Hkv]")
    B = context_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [B, MB] and context_lens [B]")
    if start is None and R != B:
        raise ValueError("without query_start there is one query row for each sequence")
    _check("pa_select_blocks", _sparse_fn("pa_select_blocks")(
        selected_tables.data_ptr(), selected_lens.data_ptr(), query.data_ptr(), bounds.data_ptr(),
        bound_scales.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
        # (no rows: empty tensors have no address)
        context_lens.data_ptr(), start, B, int(max_q_len) if R else 0, Hq, Hkv, d,
        int(block_size), NB, int(max_context_len), picked[2], int(num_sink), int(num_recent),
        _dtype_code(query), _stream(stream)))
    return selected_tables, selected_lens


def _decode_sparse(name, out, query, k_cache, v_cache, selected_tables, selected_lens, scale,
                   scales, stream):
    dev = _device_of("query", query)
    dtype = query.dtype
    cache = _U8 if scales else dtype
    _all_fit(dev, query=(query, dtype), out=(out, dtype), k_cache=(k_cache, cache),
             v_cache=(v_cache, cache), selected_tables=(selected_tables, _I32),
             selected_lens=(selected_lens, _I32))
    picked = selected_tables.shape
    if query.dim() != 3 or out.shape != query.shape:
        raise ValueError("query and out must be [R, Hq, d], alike")
    R, Hq, d = query.shape
    NB, Hkv, bs = _cache_shape(name, k_cache, d)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    if len(picked) != 3 or picked[:2] != (R, Hkv) or selected_lens.shape != picked[:2]:
        raise ValueError("selected_tables must be [R, Hkv, K] and selected_lens [R, Hkv]")
    _check(name, _sparse_fn(name)(
        out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        selected_tables.data_ptr(), selected_lens.data_ptr(), R, picked[2], Hq, Hkv, d, bs, NB,
        float(scale), *scales, _dtype_code(query), _stream(stream)))
    return out


def pa_decode_sparse(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, selected_tables: torch.Tensor,
                     selected_lens: torch.Tensor, scale: float, stream=None) -> torch.Tensor:
    """Decode attention of query [R, Hq, d] into ``out``, row r and KV head g
    over the first selected_lens[r, g] tokens of the blocks
    selected_tables[r, g, :] (pa_select_blocks)."""
    st = (_bind or _native()).sparse(0, out, query, k_cache, v_cache, selected_tables,
                                     selected_lens, scale, 1.0, 1.0, stream)
    if st == 0:
        return out
    if st > 0:
        raise PaError("pa_decode_sparse", st)
    return _decode_sparse("pa_decode_sparse", out, query, k_cache, v_cache, selected_tables,
                          selected_lens, scale, (), stream)


def pa_decode_sparse_fp8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, selected_tables: torch.Tensor,
                         selected_lens: torch.Tensor, scale: float, k_scale: float,
                         v_scale: float, stream=None) -> torch.Tensor:
    """pa_decode_sparse over uint8 FP8 E4M3 caches, fp16 or bf16 queries and output."""
    st = (_bind or _native()).sparse(1, out, query, k_cache, v_cache, selected_tables,
                                     selected_lens, scale, k_scale, v_scale, stream)
    if st == 0:
        return out
    if st > 0:
        raise PaError("pa_decode_sparse_fp8", st)
    return _decode_sparse("pa_decode_sparse_fp8", out, query, k_cache, v_cache, selected_tables,
                          selected_lens, scale, (float(k_scale), float(v_scale)), stream)


def pa_decode_sparse_fp4(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, selected_tables: torch.Tensor,
                         selected_lens: torch.Tensor, scale: float, k_scale: float,
                         v_scale: float, stream=None) -> torch.Tensor:
    """pa_decode_sparse over FP4 caches, fp16 or bf16 queries and output."""
    st = (_bind or _native()).sparse(2, out, query, k_cache, v_cache, selected_tables,
                                     selected_lens, scale, k_scale, v_scale, stream)
    if st == 0:
        return out
    if st > 0:
        raise PaError("pa_decode_sparse_fp4", st)
    return _decode_sparse("pa_decode_sparse_fp4", out, query, k_cache, v_cache, selected_tables,
                          selected_lens, scale, (float(k_scale), float(v_scale)), stream)


def pa_selftest_bounded_wait(stream=None) -> None:
    """Launch the wait-limit self-test: one CTA waits on a barrier nothing
    completes, gives up after about a second and sets DEVERR_TIMEOUT."""
    _check("pa_selftest_bounded_wait", _load().pa_selftest_bounded_wait(_stream(stream)))


def pa_device_errors(stream=None) -> int:
    """Wait for ``stream`` and return (and clear) the device error bits."""
    flags = ctypes.c_uint32(0)
    _check("pa_device_errors", _load().pa_device_errors(_stream(stream), ctypes.byref(flags)))
    return int(flags.value)
