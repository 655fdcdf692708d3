"""Thin ctypes binding of libpagedkv.so (C ABI: include/pagedkv.h).

The functions carry the ABI's names and only marshal arguments: torch
tensors become device pointers and the current CUDA stream becomes the
stream handle. Every computation runs in the library's kernels. There is no
CPU path: if the library is missing or the device is not an sm_103 GPU, the
call raises.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import build as _build

c_i32, c_i64, c_u32, c_void_p, c_size_t, c_float = (
    ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t,
    ctypes.c_float)

PKV_OK = 0
PKV_ERR_SCRATCH_LIMIT = -8
DEVERR_SLOT_RANGE = 0x1
DEVERR_BLOCK_RANGE = 0x2
DEVERR_LENGTHS = 0x4
DEVERR_TIMEOUT = 0x8
DEVERR_SHARED = 0x10
DEVERR_NO_BLOCKS = 0x20
DEVERR_REF_COUNT = 0x40
DEVERR_CHUNK_KEYS = 0x80


class pkv_cache_layout(ctypes.Structure):
    _fields_ = [("num_blocks", c_i32), ("block_size", c_i32), ("num_kv_heads", c_i32),
                ("head_dim", c_i32)]


PKV_TRACE_EVENTS = 5


PKV_OPTIONS_SCORES = 1
PKV_OPTIONS_FEW_ROWS = 1


class pkv_score_options(ctypes.Structure):
    _fields_ = [("softcap", c_float), ("alibi_slopes", c_void_p), ("key_begin", c_void_p),
                ("key_end", c_void_p), ("reserved", c_i32 * 4)]


class pkv_attention_options(ctypes.Structure):
    _fields_ = [("decode_splits", c_i32), ("shared_prefix_len", c_i32),
                ("shared_first_req", c_i32), ("shared_num_reqs", c_i32),
                ("reserved", c_i32 * 4), ("trace_events", ctypes.POINTER(c_void_p)),
                ("scores", ctypes.POINTER(pkv_score_options))]


_SIGNATURES = {
    "pkv_abi_version": (c_i32, []),
    "pkv_status_string": (ctypes.c_char_p, [c_i32]),
    "pkv_last_cuda_error": (ctypes.c_char_p, []),
    "pkv_slot_mapping": (c_i32, [c_void_p, c_void_p, c_i32, c_void_p, c_void_p, c_i32, c_i32,
                                 c_i32, c_i32, c_void_p]),
    "pkv_paged_kv_write": (c_i32, [c_void_p, c_void_p, c_void_p, c_i64, c_i64, c_void_p, c_i32,
                                   pkv_cache_layout, c_void_p]),
    "pkv_attention_workspace_size": (c_i64, [c_i32, c_i32, pkv_cache_layout,
                                             ctypes.POINTER(pkv_attention_options)]),
    "pkv_paged_attention": (c_i32, [c_void_p, c_void_p, c_i64, c_void_p, c_void_p, c_i32,
                                    c_void_p, c_void_p, c_void_p, c_i32, c_i32, c_i32, c_i32,
                                    c_i32, c_float, pkv_cache_layout, c_void_p, c_size_t,
                                    ctypes.POINTER(pkv_attention_options), c_void_p]),
    "pkv_get_device_errors": (c_i32, [ctypes.POINTER(c_u32), c_i32, c_void_p]),
    "pkv_copy_blocks": (c_i32, [c_void_p, c_i32, c_void_p, c_i32, c_void_p, c_i32,
                                pkv_cache_layout, c_void_p]),
    "pkv_slot_mapping_and_write": (c_i32, [c_void_p, c_void_p, c_void_p, c_i64, c_i64, c_void_p,
                                           c_void_p, c_i32, c_void_p, c_void_p, c_i32, c_i32,
                                           pkv_cache_layout, c_void_p]),
    "pkv_paged_attention_with_write": (
        c_i32, [c_void_p, c_void_p, c_i64, c_void_p, c_void_p, c_void_p, c_i64, c_i64, c_void_p,
                c_void_p, c_i32, c_void_p, c_void_p, c_void_p, c_i32, c_i32, c_i32, c_i32, c_i32,
                c_float, pkv_cache_layout, c_void_p, c_size_t,
                ctypes.POINTER(pkv_attention_options), c_void_p]),
    "pkv_build_step_tables": (
        c_i32, [c_void_p, c_i32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_i32, c_i32,
                c_void_p, c_void_p, c_void_p, c_void_p, c_i32, c_i32, c_void_p]),
    "pkv_release_blocks": (
        c_i32, [c_void_p, c_i32, c_i32, c_void_p, c_void_p, c_i32, c_void_p, c_void_p, c_void_p,
                c_void_p, c_i32, c_i32, c_void_p, c_size_t, c_void_p]),
    "pkv_release_workspace_size": (c_i64, [c_i32, c_i32]),
    "pkv_paged_attention_static_workspace": (
        c_i32, [c_void_p, c_void_p, c_i64, c_void_p, c_void_p, c_i32, c_void_p, c_void_p,
                c_void_p, c_i32, c_i32, c_i32, c_i32, c_i32, c_float, pkv_cache_layout,
                ctypes.POINTER(pkv_attention_options), c_void_p]),
    "pkv_quant_kv_write": (c_i32, [c_void_p, c_void_p, c_void_p, c_void_p, c_i64, c_i64, c_void_p,
                                   c_i32, pkv_cache_layout, c_void_p]),
    "pkv_quant_slot_mapping_and_write": (
        c_i32, [c_void_p, c_void_p, c_void_p, c_void_p, c_i64, c_i64, c_void_p, c_void_p, c_i32,
                c_void_p, c_void_p, c_i32, c_i32, pkv_cache_layout, c_void_p]),
    "pkv_quant_kv_read": (c_i32, [c_void_p, c_void_p, c_i64, c_i64, c_void_p, c_void_p, c_void_p,
                                  c_i32, pkv_cache_layout, c_void_p]),
    "pkv_quant_copy_blocks": (c_i32, [c_void_p, c_void_p, c_i32, c_void_p, c_void_p, c_i32,
                                      c_void_p, c_i32, pkv_cache_layout, c_void_p]),
    "pkv_quant_few_rows": (c_i32, [c_i32, c_i32, c_i32]),
    "pkv_quant_attention_workspace_size": (
        c_i64, [c_i32, c_i32, c_i32, pkv_cache_layout, c_i64,
                ctypes.POINTER(pkv_attention_options)]),
    "pkv_quant_paged_attention": (
        c_i32, [c_void_p, c_void_p, c_i64, c_void_p, c_void_p, c_void_p, c_i32, c_void_p, c_void_p,
                c_void_p, c_i32, c_i32, c_i32, c_i32, c_i32, c_float, pkv_cache_layout, c_void_p,
                c_size_t, ctypes.POINTER(pkv_attention_options), c_void_p]),
    "pkv_quant_paged_attention_with_write": (
        c_i32, [c_void_p, c_void_p, c_i64, c_void_p, c_void_p, c_void_p, c_void_p, c_i64, c_i64,
                c_void_p, c_void_p, c_i32, c_void_p, c_void_p, c_void_p, c_i32, c_i32, c_i32,
                c_i32, c_i32, c_float, pkv_cache_layout, c_void_p, c_size_t,
                ctypes.POINTER(pkv_attention_options), c_void_p]),
}

_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libpagedkv.so (building it first when it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build_library()
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run paged_kv_cache_hkv_gb300.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class PagedKVError(RuntimeError):
    def __init__(self, name, status):
        lib = load()
        msg = lib.pkv_status_string(status).decode()
        extra = lib.pkv_last_cuda_error().decode()
        super().__init__(f"{name} failed: {msg} ({status})" + (f": {extra}" if extra else ""))
        self.status = status


def _check(name, status):
    if status != PKV_OK:
        raise PagedKVError(name, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _current_stream(device):
    """Raw handle of the device's current stream. torch.cuda.current_stream()
    makes an object, 3.1 us a call instead of 0.4 and half of a small call's host
    time, but is the public way: for a torch without the short one."""
    try:
        return torch._C._cuda_getCurrentRawStream(device)
    except AttributeError:
        return torch.cuda.current_stream(device).cuda_stream


def _stream(stream, device=None):
    """The stream's handle. device: index of the device that the call's tensors
    are on, where that is to be checked: the library launches on the current one."""
    if stream is None:
        current = torch.cuda.current_device()
        if device is not None and device != current:
            raise ValueError(f"tensors on cuda:{device}, the current device is cuda:{current}")
        return ctypes.c_void_p(_current_stream(current))
    if device is not None and (device != torch.cuda.current_device() or
                               device != stream.device.index):
        raise ValueError(f"tensors on cuda:{device}, a stream of {stream.device}, the current "
                         f"device is cuda:{torch.cuda.current_device()}")
    return ctypes.c_void_p(stream.cuda_stream)


def _require(t, dtype, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def layout_of(kv_cache: torch.Tensor) -> pkv_cache_layout:
    """Layout struct of a pool tensor [num_blocks, 2, block_size, Hkv, D]."""
    if kv_cache.dim() != 5 or kv_cache.shape[1] != 2 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [num_blocks, 2, block_size, Hkv, D] tensor")
    nb, _, bs, hkv, d = kv_cache.shape
    return pkv_cache_layout(nb, bs, hkv, d)


def abi_version() -> int:
    return load().pkv_abi_version()


def pkv_slot_mapping(slot_mapping, block_table, query_start_loc, num_computed_tokens,
                     num_blocks: int, block_size: int = 16, stream=None):
    """slot_mapping (int64 [T]) <- slot of each new token (see pagedkv.h)."""
    _require(slot_mapping, torch.int64, "slot_mapping")
    for t, n in ((block_table, "block_table"), (query_start_loc, "query_start_loc"),
                 (num_computed_tokens, "num_computed_tokens")):
        _require(t, torch.int32, n)
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    _check("pkv_slot_mapping", load().pkv_slot_mapping(
        _ptr(slot_mapping), _ptr(block_table), block_table.shape[1], _ptr(query_start_loc),
        _ptr(num_computed_tokens), num_computed_tokens.shape[0], slot_mapping.shape[0],
        num_blocks, block_size, _stream(stream)))
    return slot_mapping


def pkv_paged_kv_write(kv_cache, key, value, slot_mapping, stream=None):
    """Scatter key/value rows ([T, Hkv, D] bf16, row-strided allowed) into the pool."""
    for t, n in ((kv_cache, "kv_cache"), (key, "key"), (value, "value")):
        _require(t, torch.bfloat16, n)
    _require(slot_mapping, torch.int64, "slot_mapping")
    for t, n in ((key, "key"), (value, "value")):
        if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} must be [T, Hkv, D] with contiguous rows")
    lay = layout_of(kv_cache)
    _check("pkv_paged_kv_write", load().pkv_paged_kv_write(
        _ptr(kv_cache), _ptr(key), _ptr(value), key.stride(0), value.stride(0),
        _ptr(slot_mapping), key.shape[0], lay, _stream(stream)))


def pkv_slot_mapping_and_write(kv_cache, key, value, block_table, query_start_loc,
                               num_computed_tokens, slot_mapping=None, stream=None):
    """Slot mapping and cache write in one launch (see pagedkv.h). slot_mapping
    (int64 [T]) receives the slots when given."""
    for t, n in ((kv_cache, "kv_cache"), (key, "key"), (value, "value")):
        _require(t, torch.bfloat16, n)
    for t, n in ((block_table, "block_table"), (query_start_loc, "query_start_loc"),
                 (num_computed_tokens, "num_computed_tokens")):
        _require(t, torch.int32, n)
    if slot_mapping is not None:
        _require(slot_mapping, torch.int64, "slot_mapping")
    for t, n in ((key, "key"), (value, "value")):
        if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} must be [T, Hkv, D] with contiguous rows")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    lay = layout_of(kv_cache)
    _check("pkv_slot_mapping_and_write", load().pkv_slot_mapping_and_write(
        _ptr(kv_cache), _ptr(key), _ptr(value), key.stride(0), value.stride(0),
        _ptr(slot_mapping), _ptr(block_table), block_table.shape[1], _ptr(query_start_loc),
        _ptr(num_computed_tokens), num_computed_tokens.shape[0], key.shape[0], lay,
        _stream(stream)))
    return slot_mapping


def pkv_copy_blocks(dst_pool, src_pool, block_pairs, stream=None):
    """dst_pool[d] = src_pool[s] for each (s, d) row of block_pairs (int32
    [n, 2] on the device). Pools are CUDA tensors or pinned host tensors."""
    for t, n in ((dst_pool, "dst_pool"), (src_pool, "src_pool")):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{n} must be bfloat16")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{n} must be a CUDA tensor or pinned host memory")
    _require(block_pairs, torch.int32, "block_pairs")
    if block_pairs.dim() != 2 or block_pairs.shape[1] != 2 or not block_pairs.is_contiguous():
        raise ValueError("block_pairs must be a contiguous [n, 2] int32 tensor")
    lay = layout_of(src_pool)
    if tuple(dst_pool.shape[1:]) != tuple(src_pool.shape[1:]) or not dst_pool.is_contiguous():
        raise ValueError("pools must share the block shape")
    _check("pkv_copy_blocks", load().pkv_copy_blocks(
        _ptr(dst_pool), dst_pool.shape[0], _ptr(src_pool), src_pool.shape[0],
        _ptr(block_pairs), block_pairs.shape[0], lay, _stream(stream)))


def _one_device(first, *tensors):
    for t in tensors:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on {first.device} and {t.device} in one call")


def _scored_device(q, options, *tensors):
    """Device index to check a call's stream against, its other tensors being on
    q's device: scored calls only."""
    if options is None or not options.contents.scores:
        return None
    _one_device(q, *tensors)
    return q.device.index


def _scores(q, softcap, alibi_slopes, key_begin, key_end):
    """pkv_score_options of a call on q [T, Hq, D] (None when all are off)."""
    softcap = float(softcap or 0.0)
    if softcap == 0.0 and alibi_slopes is None and key_begin is None and key_end is None:
        return None
    if alibi_slopes is not None:
        _require(alibi_slopes, torch.float32, "alibi_slopes")
        if alibi_slopes.shape != (q.shape[1],) or not alibi_slopes.is_contiguous():
            raise ValueError("alibi_slopes must be a contiguous [Hq] tensor")
    for t, n in ((key_begin, "key_begin"), (key_end, "key_end")):
        if t is not None:
            _require(t, torch.int32, n)
            if t.shape != (q.shape[0],) or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous [T] tensor")
    _one_device(q, alibi_slopes, key_begin, key_end)
    o = pkv_score_options()
    o.softcap = softcap
    o.alibi_slopes, o.key_begin, o.key_end = _ptr(alibi_slopes), _ptr(key_begin), _ptr(key_end)
    o._keep = (alibi_slopes, key_begin, key_end)
    return o


def _options(decode_splits, trace_events=None, shared_prefix=None, scores=None, few_rows=None):
    """Options struct (or None for the defaults). shared_prefix: None, or
    (shared_prefix_len, shared_first_req, shared_num_reqs) -- see pagedkv.h;
    scores: None, or what _scores returns; few_rows: 8-bit pool (see
    pkv_quant_few_rows in pagedkv.h)."""
    if decode_splits is None and trace_events is None and shared_prefix is None and (
            scores is None and few_rows is None):
        return None
    o = pkv_attention_options()
    o.decode_splits = int(decode_splits or 0)
    if few_rows is not None:
        o.reserved[PKV_OPTIONS_FEW_ROWS] = int(few_rows)
    if shared_prefix is not None:
        o.shared_prefix_len, o.shared_first_req, o.shared_num_reqs = (int(x) for x in shared_prefix)
    if trace_events is not None:
        if len(trace_events) != PKV_TRACE_EVENTS:
            raise ValueError(f"trace_events needs {PKV_TRACE_EVENTS} torch.cuda.Event")
        handles = [e.cuda_event for e in trace_events]
        if not all(handles):
            raise ValueError("trace events must be created (recorded once) before use")
        arr = (c_void_p * PKV_TRACE_EVENTS)(*[c_void_p(h) for h in handles])
        o.trace_events = ctypes.cast(arr, ctypes.POINTER(c_void_p))
        o._keep = arr
    if scores is not None:
        o.reserved[0] = PKV_OPTIONS_SCORES
        o.scores = ctypes.pointer(scores)
        o._keep_scores = scores
    return ctypes.pointer(o)


def pkv_attention_workspace_size(num_reqs: int, num_q_heads: int, kv_cache,
                                 decode_splits=None, shared_prefix=None) -> int:
    """Workspace bytes for pkv_paged_attention; kv_cache is the pool tensor
    or a pkv_cache_layout."""
    lay = kv_cache if isinstance(kv_cache, pkv_cache_layout) else layout_of(kv_cache)
    n = load().pkv_attention_workspace_size(num_reqs, num_q_heads, lay,
                                            _options(decode_splits, None, shared_prefix))
    if n < 0:
        raise PagedKVError("pkv_attention_workspace_size", int(n))
    return int(n)


def pkv_paged_attention(out, q, kv_cache, block_table, seq_lens, query_start_loc,
                        num_computed_tokens, *, max_query_len: int, max_seq_len: int,
                        scale: float, workspace, decode_splits=None, trace_events=None,
                        shared_prefix=None, softcap=0.0, alibi_slopes=None, key_begin=None,
                        key_end=None, stream=None):
    """out [T, Hq, D] bf16 <- attention of one mixed step (see pagedkv.h).

    trace_events: optional list of PKV_TRACE_EVENTS torch.cuda.Event (created
    with enable_timing=True) recorded around the call's kernels.
    softcap, alibi_slopes (fp32 [Hq]), key_begin, key_end (int32 [T]): capped,
    biased or range-masked scores (pkv_score_options in pagedkv.h)."""
    for t, n in ((out, "out"), (q, "q"), (kv_cache, "kv_cache")):
        _require(t, torch.bfloat16, n)
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens"),
                 (query_start_loc, "query_start_loc"),
                 (num_computed_tokens, "num_computed_tokens")):
        _require(t, torch.int32, n)
    if not out.is_contiguous() or not block_table.is_contiguous():
        raise ValueError("out and block_table must be contiguous")
    if q.dim() != 3 or q.stride(2) != 1 or q.stride(1) != q.shape[2]:
        raise ValueError("q must be [T, Hq, D] with contiguous rows")
    lay = layout_of(kv_cache)
    options = _options(decode_splits, trace_events, shared_prefix,
                       _scores(q, softcap, alibi_slopes, key_begin, key_end))
    device = _scored_device(q, options, out, kv_cache, block_table, seq_lens, query_start_loc,
                            num_computed_tokens, workspace)
    _check("pkv_paged_attention", load().pkv_paged_attention(
        _ptr(out), _ptr(q), q.stride(0), _ptr(kv_cache), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), _ptr(query_start_loc), _ptr(num_computed_tokens),
        seq_lens.shape[0], q.shape[0], int(max_query_len), int(max_seq_len), q.shape[1],
        float(scale), lay, _ptr(workspace), workspace.numel() * workspace.element_size(),
        options, _stream(stream, device)))
    return out


def pkv_paged_attention_with_write(out, q, kv_cache, key, value, block_table, seq_lens,
                                   query_start_loc, num_computed_tokens, *, max_query_len: int,
                                   max_seq_len: int, scale: float, workspace, slot_mapping=None,
                                   decode_splits=None, trace_events=None, shared_prefix=None,
                                   softcap=0.0, alibi_slopes=None, key_begin=None, key_end=None,
                                   stream=None):
    """The step of one layer in one call: slot mapping and cache write of the
    new tokens, then attention (see pagedkv.h). slot_mapping (int64 [T])
    receives the slots when given. softcap, alibi_slopes, key_begin, key_end:
    as in pkv_paged_attention."""
    for t, n in ((out, "out"), (q, "q"), (kv_cache, "kv_cache"), (key, "key"),
                 (value, "value")):
        _require(t, torch.bfloat16, n)
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens"),
                 (query_start_loc, "query_start_loc"),
                 (num_computed_tokens, "num_computed_tokens")):
        _require(t, torch.int32, n)
    if slot_mapping is not None:
        _require(slot_mapping, torch.int64, "slot_mapping")
    if not out.is_contiguous() or not block_table.is_contiguous():
        raise ValueError("out and block_table must be contiguous")
    for t, n in ((q, "q"), (key, "key"), (value, "value")):
        if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} must be [T, H, D] with contiguous rows")
    if key.shape[0] != q.shape[0]:
        raise ValueError("key and q must have the same number of rows")
    lay = layout_of(kv_cache)
    options = _options(decode_splits, trace_events, shared_prefix,
                       _scores(q, softcap, alibi_slopes, key_begin, key_end))
    device = _scored_device(q, options, out, kv_cache, key, value, block_table, seq_lens,
                            query_start_loc, num_computed_tokens, workspace, slot_mapping)
    _check("pkv_paged_attention_with_write", load().pkv_paged_attention_with_write(
        _ptr(out), _ptr(q), q.stride(0), _ptr(kv_cache), _ptr(key), _ptr(value), key.stride(0),
        value.stride(0), _ptr(slot_mapping), _ptr(block_table), block_table.shape[1],
        _ptr(seq_lens), _ptr(query_start_loc), _ptr(num_computed_tokens), seq_lens.shape[0],
        q.shape[0], int(max_query_len), int(max_seq_len), q.shape[1], float(scale), lay,
        _ptr(workspace), workspace.numel() * workspace.element_size(),
        options, _stream(stream, device)))
    return out


def pkv_get_device_errors(clear: bool = True, stream=None) -> int:
    """Synchronise and read (optionally clear) the sticky device error bits."""
    v = c_u32(0)
    _check("pkv_get_device_errors",
           load().pkv_get_device_errors(ctypes.byref(v), int(clear), _stream(stream)))
    return int(v.value)


def pkv_paged_attention_static_workspace(out, q, kv_cache, block_table, seq_lens,
                                         query_start_loc, num_computed_tokens, *,
                                         max_query_len: int, max_seq_len: int, scale: float,
                                         decode_splits=None, shared_prefix=None, softcap=0.0,
                                         alibi_slopes=None, key_begin=None, key_end=None,
                                         stream=None):
    """pkv_paged_attention without a caller workspace: for callers that cannot
    allocate device memory, the library uses its built-in scratch array (see
    pagedkv.h for the size limit and the one-stream rule)."""
    for t, n in ((out, "out"), (q, "q"), (kv_cache, "kv_cache")):
        _require(t, torch.bfloat16, n)
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens"),
                 (query_start_loc, "query_start_loc"),
                 (num_computed_tokens, "num_computed_tokens")):
        _require(t, torch.int32, n)
    if not out.is_contiguous() or not block_table.is_contiguous():
        raise ValueError("out and block_table must be contiguous")
    if q.dim() != 3 or q.stride(2) != 1 or q.stride(1) != q.shape[2]:
        raise ValueError("q must be [T, Hq, D] with contiguous rows")
    options = _options(decode_splits, None, shared_prefix,
                       _scores(q, softcap, alibi_slopes, key_begin, key_end))
    device = _scored_device(q, options, out, kv_cache, block_table, seq_lens, query_start_loc,
                            num_computed_tokens)
    _check("pkv_paged_attention_static_workspace", load().pkv_paged_attention_static_workspace(
        _ptr(out), _ptr(q), q.stride(0), _ptr(kv_cache), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), _ptr(query_start_loc), _ptr(num_computed_tokens),
        seq_lens.shape[0], q.shape[0], int(max_query_len), int(max_seq_len), q.shape[1],
        float(scale), layout_of(kv_cache), options,
        _stream(stream, device)))
    return out


def _table_args(block_table, free_queue, free_state, free_state_out, ref_cnt):
    """Checks of the arguments that pkv_build_step_tables and
    pkv_release_blocks share; returns free_state_out (free_state when None)."""
    if free_state_out is None:
        free_state_out = free_state
    for t, n in ((block_table, "block_table"), (free_queue, "free_queue"),
                 (free_state, "free_state"), (free_state_out, "free_state_out"),
                 (ref_cnt, "ref_cnt")):
        if t is None and n == "ref_cnt":
            continue
        _require(t, torch.int32, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _one_device(block_table, free_queue, free_state, free_state_out, ref_cnt)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [num_reqs, max_blocks]")
    for t, n in ((free_state, "free_state"), (free_state_out, "free_state_out")):
        if t.shape != (2,):
            raise ValueError(f"{n} must be [2]: head and count")
    if free_queue.dim() != 1 or (ref_cnt is not None and ref_cnt.shape != free_queue.shape):
        raise ValueError("free_queue and ref_cnt must be [num_blocks]")
    return free_state_out


def _build_args(block_table, query_start_loc, seq_lens, slot_mapping, num_computed_tokens,
                query_lens, free_queue, free_state, free_state_out, ref_cnt, block_size,
                num_tokens):
    free_state_out = _table_args(block_table, free_queue, free_state, free_state_out, ref_cnt)
    R = block_table.shape[0]
    for t, n, size in ((query_start_loc, "query_start_loc", R + 1), (seq_lens, "seq_lens", R),
                       (num_computed_tokens, "num_computed_tokens", R),
                       (query_lens, "query_lens", R)):
        _require(t, torch.int32, n)
        if t.shape != (size,) or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous [{size}] tensor")
    if slot_mapping is not None:
        _require(slot_mapping, torch.int64, "slot_mapping")
        if slot_mapping.dim() != 1 or not slot_mapping.is_contiguous():
            raise ValueError("slot_mapping must be a contiguous [T] tensor")
        num_tokens = slot_mapping.shape[0]
    elif num_tokens is None:
        raise ValueError("num_tokens is needed without a slot_mapping")
    _one_device(block_table, query_start_loc, seq_lens, slot_mapping, num_computed_tokens,
                query_lens)
    return (_ptr(block_table), block_table.shape[1], _ptr(query_start_loc), _ptr(seq_lens),
            _ptr(slot_mapping), _ptr(num_computed_tokens), _ptr(query_lens), R, int(num_tokens),
            _ptr(free_queue), _ptr(free_state), _ptr(free_state_out), _ptr(ref_cnt),
            free_queue.shape[0], int(block_size))


def pkv_release_workspace_size(num_released: int, max_blocks_per_req: int) -> int:
    """Workspace bytes for pkv_release_blocks (0 for small releases)."""
    n = load().pkv_release_workspace_size(num_released, max_blocks_per_req)
    if n < 0:
        raise PagedKVError("pkv_release_workspace_size", int(n))
    return int(n)


def _release_args(block_table, release_rows, release_tokens, free_queue, free_state,
                  free_state_out, ref_cnt, block_size, workspace):
    if ref_cnt is None:
        raise ValueError("a release needs ref_cnt")
    free_state_out = _table_args(block_table, free_queue, free_state, free_state_out, ref_cnt)
    for t, n in ((release_rows, "release_rows"), (release_tokens, "release_tokens")):
        _require(t, torch.int32, n)
        if t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous 1-D tensor")
    if release_tokens.shape[0] != block_table.shape[0]:
        raise ValueError("release_tokens must be [num_reqs]")
    _one_device(block_table, release_rows, release_tokens, workspace)
    return (_ptr(block_table), block_table.shape[1], block_table.shape[0], _ptr(release_rows),
            _ptr(release_tokens), release_rows.shape[0], _ptr(free_queue), _ptr(free_state),
            _ptr(free_state_out), _ptr(ref_cnt), free_queue.shape[0], int(block_size),
            _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())


def pkv_build_step_tables(block_table, query_start_loc, seq_lens, slot_mapping,
                          num_computed_tokens, query_lens, free_queue, free_state, *,
                          block_size: int, ref_cnt=None, free_state_out=None, num_tokens=None,
                          stream=None):
    """One step's block tables, row starts, lengths and slots from the
    requests' lengths and the free queue (see pagedkv.h). slot_mapping (int64
    [T]) may be None when num_tokens is given; free_state_out defaults to
    free_state (in place)."""
    _check("pkv_build_step_tables", load().pkv_build_step_tables(
        *_build_args(block_table, query_start_loc, seq_lens, slot_mapping, num_computed_tokens,
                     query_lens, free_queue, free_state, free_state_out, ref_cnt, block_size,
                     num_tokens), _stream(stream, block_table.device.index)))


def pkv_release_blocks(block_table, release_rows, release_tokens, free_queue, free_state, ref_cnt,
                       *, block_size: int, workspace=None, free_state_out=None, stream=None):
    """Give back the blocks of the rows release_rows (see pagedkv.h). workspace:
    pkv_release_workspace_size() bytes, None where that is 0."""
    _check("pkv_release_blocks", load().pkv_release_blocks(
        *_release_args(block_table, release_rows, release_tokens, free_queue, free_state,
                       free_state_out, ref_cnt, block_size, workspace),
        _stream(stream, block_table.device.index)))


# (a struct of its fields alone, which no call changes)
_layout_struct = functools.lru_cache(maxsize=64)(pkv_cache_layout)


def _quant_pool(kv_cache, kv_scales, names=("kv_cache", "kv_scales"), pinned=False):
    """Layout and device index of an 8-bit pool: codes [num_blocks, 2, B, Hkv, D]
    e4m3 and their scales [num_blocks, 2, B, Hkv] uint8. (The checks of these calls
    look at each property once: they are most of a small call's host time.)"""
    for t, dtype, n in ((kv_cache, torch.float8_e4m3fn, names[0]),
                        (kv_scales, torch.uint8, names[1])):
        if t.dtype != dtype:
            raise ValueError(f"{n} must be {dtype}, got {t.dtype}")
        if not t.is_cuda and not (pinned and t.is_pinned()):
            raise ValueError(f"{n} must be a CUDA tensor" +
                             (" or pinned host memory" if pinned else ""))
    shape = kv_cache.shape
    if len(shape) != 5 or shape[1] != 2 or not kv_cache.is_contiguous():
        raise ValueError(f"{names[0]} must be a contiguous [num_blocks, 2, block_size, Hkv, D] tensor")
    nb, _, bs, hkv, d = shape
    if kv_scales.shape != (nb, 2, bs, hkv) or not kv_scales.is_contiguous():
        raise ValueError(f"{names[1]} must be a contiguous [num_blocks, 2, block_size, Hkv] tensor")
    device = kv_cache.get_device()
    if kv_scales.get_device() != device:
        raise ValueError(f"tensors on {kv_cache.device} and {kv_scales.device} in one call")
    return _layout_struct(nb, bs, hkv, d), device


def _quant_rows(t, n, num_tokens, heads, dim, device):
    """Checks of rows [T, H, D] bf16, contiguous within a token (heads None: any
    number of them); returns their row stride, 0 for a single row, whose says nothing."""
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{n} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{n} is on {t.device}, the call's pool on cuda:{device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]) or (
            num_tokens > 1 and stride[0] < shape[1] * shape[2]):
        raise ValueError(f"{n} must be [T, H, D] with contiguous rows")
    if shape[0] != num_tokens or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{n} has shape {tuple(shape)}: {num_tokens} rows of the pool's "
                         "heads and dims are wanted")
    return stride[0] if num_tokens > 1 else 0


def _quant_slots(slot_mapping, num_tokens, device):
    if slot_mapping.dtype != torch.int64 or slot_mapping.get_device() != device:
        raise ValueError(f"slot_mapping must be torch.int64 on cuda:{device}, got "
                         f"{slot_mapping.dtype} on {slot_mapping.device}")
    if slot_mapping.shape != (num_tokens,) or not slot_mapping.is_contiguous():
        raise ValueError(f"slot_mapping must be a contiguous [{num_tokens}] tensor")
    return slot_mapping.data_ptr()


def pkv_quant_kv_write(kv_cache, kv_scales, key, value, slot_mapping, stream=None):
    """Quantise key/value rows ([T, Hkv, D] bf16, row-strided allowed) into the
    8-bit pool at their slots (see pagedkv.h)."""
    lay, device = _quant_pool(kv_cache, kv_scales)
    T = key.shape[0]
    ks = _quant_rows(key, "key", T, lay.num_kv_heads, lay.head_dim, device)
    vs = _quant_rows(value, "value", T, lay.num_kv_heads, lay.head_dim, device)
    status = load().pkv_quant_kv_write(
        kv_cache.data_ptr(), kv_scales.data_ptr(), key.data_ptr(), value.data_ptr(), ks, vs,
        _quant_slots(slot_mapping, T, device), T, lay, _stream(stream, device))
    if status:
        raise PagedKVError("pkv_quant_kv_write", status)


def _quant_batch(device, block_table, query_start_loc, num_computed_tokens, seq_lens=None):
    for t, n in ((block_table, "block_table"), (query_start_loc, "query_start_loc"),
                 (num_computed_tokens, "num_computed_tokens"), (seq_lens, "seq_lens")):
        if t is None and n == "seq_lens":
            continue
        _require(t, torch.int32, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
        if t.get_device() != device:
            raise ValueError(f"{n} is on {t.device}, the call's pool on cuda:{device}")
    R = num_computed_tokens.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] != R or query_start_loc.shape != (R + 1,) or (
            num_computed_tokens.dim() != 1 or (seq_lens is not None and seq_lens.shape != (R,))):
        raise ValueError("block_table, query_start_loc, seq_lens and num_computed_tokens must be "
                         "[R, max_blocks], [R + 1], [R] and [R]")
    return R


def pkv_quant_slot_mapping_and_write(kv_cache, kv_scales, key, value, block_table, query_start_loc,
                                     num_computed_tokens, slot_mapping=None, stream=None):
    """Slot mapping and quantised cache write in one launch (see pagedkv.h).
    slot_mapping (int64 [T]) receives the slots when given."""
    lay, device = _quant_pool(kv_cache, kv_scales)
    T = key.shape[0]
    ks = _quant_rows(key, "key", T, lay.num_kv_heads, lay.head_dim, device)
    vs = _quant_rows(value, "value", T, lay.num_kv_heads, lay.head_dim, device)
    slots = None if slot_mapping is None else _quant_slots(slot_mapping, T, device)
    R = _quant_batch(device, block_table, query_start_loc, num_computed_tokens)
    _check("pkv_quant_slot_mapping_and_write", load().pkv_quant_slot_mapping_and_write(
        _ptr(kv_cache), _ptr(kv_scales), _ptr(key), _ptr(value), ks, vs, slots, _ptr(block_table),
        block_table.shape[1], _ptr(query_start_loc), _ptr(num_computed_tokens), R, T, lay,
        _stream(stream, device)))
    return slot_mapping


def pkv_quant_kv_read(key, value, kv_cache, kv_scales, slot_mapping, stream=None):
    """key, value ([T, Hkv, D] bf16, row-strided allowed) <- the pool's rows at
    the slots; rows with a negative slot stay as they are (see pagedkv.h)."""
    lay, device = _quant_pool(kv_cache, kv_scales)
    T = key.shape[0]
    ks = _quant_rows(key, "key", T, lay.num_kv_heads, lay.head_dim, device)
    vs = _quant_rows(value, "value", T, lay.num_kv_heads, lay.head_dim, device)
    status = load().pkv_quant_kv_read(
        key.data_ptr(), value.data_ptr(), ks, vs, kv_cache.data_ptr(), kv_scales.data_ptr(),
        _quant_slots(slot_mapping, T, device), T, lay, _stream(stream, device))
    if status:
        raise PagedKVError("pkv_quant_kv_read", status)


def pkv_quant_copy_blocks(dst_pool, dst_scales, src_pool, src_scales, block_pairs, stream=None):
    """Codes and scales of dst block d = those of src block s for each (s, d) row
    of block_pairs (int32 [n, 2] on the device). Pools are CUDA tensors or pinned
    host tensors."""
    _quant_pool(dst_pool, dst_scales, ("dst_pool", "dst_scales"), pinned=True)
    lay, _ = _quant_pool(src_pool, src_scales, ("src_pool", "src_scales"), pinned=True)
    _require(block_pairs, torch.int32, "block_pairs")
    if block_pairs.dim() != 2 or block_pairs.shape[1] != 2 or not block_pairs.is_contiguous():
        raise ValueError("block_pairs must be a contiguous [n, 2] int32 tensor")
    if dst_pool.shape[1:] != src_pool.shape[1:]:
        raise ValueError("pools must share the block shape")
    _one_device(block_pairs, *(t for t in (dst_pool, dst_scales, src_pool, src_scales) if t.is_cuda))
    _check("pkv_quant_copy_blocks", load().pkv_quant_copy_blocks(
        _ptr(dst_pool), _ptr(dst_scales), dst_pool.shape[0], _ptr(src_pool), _ptr(src_scales),
        src_pool.shape[0], _ptr(block_pairs), block_pairs.shape[0], lay,
        _stream(stream, block_pairs.device.index)))


def pkv_quant_few_rows(max_query_len: int, num_q_heads: int, num_kv_heads: int) -> int:
    """Most new tokens of a request that attention over the 8-bit pool takes on
    its decode kernels (see pagedkv.h)."""
    n = load().pkv_quant_few_rows(max_query_len, num_q_heads, num_kv_heads)
    if n < 0:
        raise PagedKVError("pkv_quant_few_rows", int(n))
    return int(n)


def quant_chunk_keys(query_lens, seq_lens, group: int, block_size: int, few_rows=None,
                     max_query_len=None) -> int:
    """chunk_keys of pkv_quant_attention_workspace_size for a step of these (host)
    lengths; group: q heads per kv head; few_rows, max_query_len: as in the attention
    call (the longest of query_lens where not given)."""
    if max_query_len is None:
        max_query_len = max(query_lens, default=0)
    few = few_rows or pkv_quant_few_rows(max_query_len, group, 1)
    return sum(-(-L // block_size) * block_size for n, L in zip(query_lens, seq_lens) if n > few)


def pkv_quant_attention_workspace_size(num_reqs: int, num_q_heads: int, kv_cache, *,
                                       max_blocks_per_req: int, chunk_keys: int,
                                       decode_splits=None, shared_prefix=None) -> int:
    """Workspace bytes for pkv_quant_paged_attention (see pagedkv.h; chunk_keys:
    see quant_chunk_keys); kv_cache is the codes' tensor or a pkv_cache_layout."""
    lay = kv_cache if isinstance(kv_cache, pkv_cache_layout) else layout_of(kv_cache)
    n = load().pkv_quant_attention_workspace_size(
        num_reqs, max_blocks_per_req, num_q_heads, lay, int(chunk_keys),
        _options(decode_splits, None, shared_prefix))
    if n < 0:
        raise PagedKVError("pkv_quant_attention_workspace_size", int(n))
    return int(n)


def _quant_attention_args(out, q, kv_cache, kv_scales, block_table, seq_lens, query_start_loc,
                          num_computed_tokens, max_query_len, max_seq_len, scale, workspace,
                          options, write=None):
    """Checked and marshalled arguments of pkv_quant_paged_attention, or with
    write = (key, value, slot_mapping) of its _with_write form; all but the stream."""
    lay, device = _quant_pool(kv_cache, kv_scales)
    T = q.shape[0]
    qs = _quant_rows(q, "q", T, None, lay.head_dim, device)
    _require(out, torch.bfloat16, "out")
    if out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous and of q's shape")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    R = _quant_batch(device, block_table, query_start_loc, num_computed_tokens, seq_lens)
    _one_device(kv_cache, out, workspace)
    rows = ()
    if write is not None:
        key, value, slot_mapping = write
        ks = _quant_rows(key, "key", T, lay.num_kv_heads, lay.head_dim, device)
        vs = _quant_rows(value, "value", T, lay.num_kv_heads, lay.head_dim, device)
        rows = (_ptr(key), _ptr(value), ks, vs,
                None if slot_mapping is None else _quant_slots(slot_mapping, T, device))
    return (_ptr(out), _ptr(q), qs, _ptr(kv_cache), _ptr(kv_scales), *rows,
            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), _ptr(query_start_loc),
            _ptr(num_computed_tokens), R, T, int(max_query_len), int(max_seq_len), q.shape[1],
            float(scale), lay, _ptr(workspace), workspace.numel() * workspace.element_size(),
            options)


def pkv_quant_paged_attention(out, q, kv_cache, kv_scales, block_table, seq_lens, query_start_loc,
                              num_computed_tokens, *, max_query_len: int, max_seq_len: int,
                              scale: float, workspace, decode_splits=None, trace_events=None,
                              shared_prefix=None, softcap=0.0, alibi_slopes=None, key_begin=None,
                              key_end=None, few_rows=None, stream=None):
    """out [T, Hq, D] bf16 <- attention of one mixed step over the 8-bit pool (see
    pagedkv.h); options as in pkv_paged_attention. few_rows: the most new tokens of a
    request that goes on the decode kernels, where the default (pkv_quant_few_rows)
    is not wanted."""
    options = _options(decode_splits, trace_events, shared_prefix,
                       _scores(q, softcap, alibi_slopes, key_begin, key_end), few_rows)
    _check("pkv_quant_paged_attention", load().pkv_quant_paged_attention(
        *_quant_attention_args(out, q, kv_cache, kv_scales, block_table, seq_lens,
                               query_start_loc, num_computed_tokens, max_query_len, max_seq_len,
                               scale, workspace, options), _stream(stream, q.device.index)))
    return out


def pkv_quant_paged_attention_with_write(out, q, kv_cache, kv_scales, key, value, block_table,
                                         seq_lens, query_start_loc, num_computed_tokens, *,
                                         max_query_len: int, max_seq_len: int, scale: float,
                                         workspace, slot_mapping=None, decode_splits=None,
                                         trace_events=None, shared_prefix=None, softcap=0.0,
                                         alibi_slopes=None, key_begin=None, key_end=None,
                                         few_rows=None, stream=None):
    """The step of one layer on the 8-bit pool in one call: slot mapping and
    quantised write of the new tokens, then attention (see pagedkv.h;
    few_rows: as in pkv_quant_paged_attention)."""
    options = _options(decode_splits, trace_events, shared_prefix,
                       _scores(q, softcap, alibi_slopes, key_begin, key_end), few_rows)
    _check("pkv_quant_paged_attention_with_write", load().pkv_quant_paged_attention_with_write(
        *_quant_attention_args(out, q, kv_cache, kv_scales, block_table, seq_lens,
                               query_start_loc, num_computed_tokens, max_query_len, max_seq_len,
                               scale, workspace, options, (key, value, slot_mapping)),
        _stream(stream, q.device.index)))
    return out


class TableCalls:
    """pkv_build_step_tables and pkv_release_blocks on buffers that a serving
    loop keeps, with their arguments checked and marshalled once (as StepCalls
    does for the step's calls). Pass the arguments of either call or of both; the
    release's workspace is made here. Like the tensors, it has to live until the
    last call has finished: keep the object for as long."""

    def __init__(self, *, block_table, free_queue, free_state, block_size: int, ref_cnt=None,
                 free_state_out=None, query_start_loc=None, seq_lens=None, slot_mapping=None,
                 num_computed_tokens=None, query_lens=None, num_tokens=None, release_rows=None,
                 release_tokens=None):
        self.lib = load()
        self.build_args = self.release_args = None
        if query_lens is not None:
            self.build_args = _build_args(
                block_table, query_start_loc, seq_lens, slot_mapping, num_computed_tokens,
                query_lens, free_queue, free_state, free_state_out, ref_cnt, block_size,
                num_tokens)
        workspace = None
        if release_rows is not None:
            nbytes = pkv_release_workspace_size(release_rows.shape[0], block_table.shape[1])
            if nbytes:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=block_table.device)
            self.release_args = _release_args(block_table, release_rows, release_tokens,
                                              free_queue, free_state, free_state_out, ref_cnt,
                                              block_size, workspace)
        self._device = block_table.device.index
        if self.build_args is None and self.release_args is None:
            raise ValueError("pass query_lens (build), release_rows (release) or both")
        # the tensors stay referenced, so their memory stays valid
        self._keep = (block_table, free_queue, free_state, ref_cnt, free_state_out,
                      query_start_loc, seq_lens, slot_mapping, num_computed_tokens, query_lens,
                      release_rows, release_tokens, workspace)

    def build(self, stream=None):
        if self.build_args is None:
            raise ValueError("these TableCalls were made without query_lens")
        status = self.lib.pkv_build_step_tables(*self.build_args,
                                                _stream(stream, self._device))
        if status:
            raise PagedKVError("pkv_build_step_tables", status)

    def release(self, stream=None):
        if self.release_args is None:
            raise ValueError("these TableCalls were made without release_rows")
        status = self.lib.pkv_release_blocks(*self.release_args,
                                             _stream(stream, self._device))
        if status:
            raise PagedKVError("pkv_release_blocks", status)


class StepCalls:
    """The calls of one step -- pkv_slot_mapping, pkv_paged_kv_write,
    pkv_paged_attention; with fused_write pkv_slot_mapping_and_write then
    pkv_paged_attention; with write_in_attention the one call
    pkv_paged_attention_with_write -- with their arguments checked and
    marshalled once.

    A serving loop that keeps its step buffers (as DeviceStep does) pays the
    argument checks and the tensor-to-pointer conversion once, not on every
    step; ``run`` then makes the three C calls in a row on the given stream.
    The buffers must stay allocated and keep their shapes while the object is
    used. With kv_scales the pool is the 8-bit one and the calls are the
    pkv_quant_ ones."""

    def __init__(self, *, slot_mapping, block_table, query_start_loc, num_computed_tokens,
                 kv_cache, key, value, out, q, seq_lens, max_query_len: int,
                 max_seq_len: int, scale: float, workspace, decode_splits=None,
                 shared_prefix=None, fused_write=False, write_in_attention=False, softcap=0.0,
                 alibi_slopes=None, key_begin=None, key_end=None, kv_scales=None,
                 few_rows=None):
        self.fused_write = bool(fused_write)
        self.write_in_attention = bool(write_in_attention)
        self._write, self._mapped_write, self._attend, self._attend_write = (
            ("pkv_quant_kv_write", "pkv_quant_slot_mapping_and_write",
             "pkv_quant_paged_attention", "pkv_quant_paged_attention_with_write")
            if kv_scales is not None else
            ("pkv_paged_kv_write", "pkv_slot_mapping_and_write", "pkv_paged_attention",
             "pkv_paged_attention_with_write"))
        # the tensors stay referenced, so their memory stays valid
        self._keep = (slot_mapping, block_table, query_start_loc, num_computed_tokens,
                      kv_cache, key, value, out, q, seq_lens, workspace, kv_scales)
        self._write_device = None if kv_scales is None else kv_cache.device.index
        if kv_scales is not None:
            self._marshal_quant(slot_mapping, block_table, query_start_loc, num_computed_tokens,
                                kv_cache, kv_scales, key, value, out, q, seq_lens, max_query_len,
                                max_seq_len, scale, workspace,
                                _options(decode_splits, None, shared_prefix,
                                         _scores(q, softcap, alibi_slopes, key_begin, key_end),
                                         few_rows))
            return
        if few_rows is not None:
            raise ValueError("few_rows is for the 8-bit pool (kv_scales)")
        _require(slot_mapping, torch.int64, "slot_mapping")
        for t, n in ((block_table, "block_table"), (query_start_loc, "query_start_loc"),
                     (num_computed_tokens, "num_computed_tokens"), (seq_lens, "seq_lens")):
            _require(t, torch.int32, n)
        for t, n in ((kv_cache, "kv_cache"), (key, "key"), (value, "value"), (out, "out"),
                     (q, "q")):
            _require(t, torch.bfloat16, n)
        for t, n in ((key, "key"), (value, "value"), (q, "q")):
            if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
                raise ValueError(f"{n} must be [T, H, D] with contiguous rows")
        if not out.is_contiguous() or not block_table.is_contiguous():
            raise ValueError("out and block_table must be contiguous")
        lay = layout_of(kv_cache)
        self.lib = load()
        self._opts = _options(decode_splits, None, shared_prefix,
                              _scores(q, softcap, alibi_slopes, key_begin, key_end))
        self._device = _scored_device(q, self._opts, out, kv_cache, key, value, block_table,
                                      seq_lens, query_start_loc, num_computed_tokens, workspace,
                                      slot_mapping)
        self.slot_args = (
            _ptr(slot_mapping), _ptr(block_table), block_table.shape[1], _ptr(query_start_loc),
            _ptr(num_computed_tokens), num_computed_tokens.shape[0], slot_mapping.shape[0],
            lay.num_blocks, lay.block_size)
        self.write_args = (
            _ptr(kv_cache), _ptr(key), _ptr(value), key.stride(0), value.stride(0),
            _ptr(slot_mapping), key.shape[0], lay)
        if self.write_in_attention and key.shape[0] != q.shape[0]:
            raise ValueError("key and q must have the same number of rows")
        self.mapped_write_args = (
            _ptr(kv_cache), _ptr(key), _ptr(value), key.stride(0), value.stride(0),
            _ptr(slot_mapping), _ptr(block_table), block_table.shape[1], _ptr(query_start_loc),
            _ptr(num_computed_tokens), num_computed_tokens.shape[0], key.shape[0], lay)
        self.attn_args = (
            _ptr(out), _ptr(q), q.stride(0), _ptr(kv_cache), _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), _ptr(query_start_loc),
            _ptr(num_computed_tokens), seq_lens.shape[0], q.shape[0], int(max_query_len),
            int(max_seq_len), q.shape[1], float(scale), lay, _ptr(workspace),
            workspace.numel() * workspace.element_size(), self._opts)
        self.attn_write_args = (
            _ptr(out), _ptr(q), q.stride(0), _ptr(kv_cache), _ptr(key), _ptr(value),
            key.stride(0), value.stride(0), _ptr(slot_mapping), _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), _ptr(query_start_loc),
            _ptr(num_computed_tokens), seq_lens.shape[0], q.shape[0], int(max_query_len),
            int(max_seq_len), q.shape[1], float(scale), lay, _ptr(workspace),
            workspace.numel() * workspace.element_size(), self._opts)

    def _marshal_quant(self, slot_mapping, block_table, query_start_loc, num_computed_tokens,
                       kv_cache, kv_scales, key, value, out, q, seq_lens, max_query_len,
                       max_seq_len, scale, workspace, options):
        """The arguments of the 8-bit pool's calls (kv_scales given)."""
        self.lib = load()
        self._opts = options
        self._device = kv_cache.device.index
        args = (out, q, kv_cache, kv_scales, block_table, seq_lens, query_start_loc,
                num_computed_tokens, max_query_len, max_seq_len, scale, workspace, options)
        self.attn_args = _quant_attention_args(*args)
        self.attn_write_args = _quant_attention_args(*args, (key, value, slot_mapping))
        lay, T, R = layout_of(kv_cache), q.shape[0], num_computed_tokens.shape[0]
        ks, vs = (_quant_rows(t, n, T, lay.num_kv_heads, lay.head_dim, self._device)
                  for t, n in ((key, "key"), (value, "value")))
        rows = (_ptr(kv_cache), _ptr(kv_scales), _ptr(key), _ptr(value), ks, vs,
                _quant_slots(slot_mapping, T, self._device))
        tables = (_ptr(block_table), block_table.shape[1], _ptr(query_start_loc),
                  _ptr(num_computed_tokens), R, T)
        self.slot_args = (_ptr(slot_mapping), *tables, lay.num_blocks, lay.block_size)
        self.write_args = (*rows, T, lay)
        self.mapped_write_args = (*rows, *tables, lay)

    def slot_map(self, stream=None):
        self._call("pkv_slot_mapping", self.slot_args, _stream(stream, self._write_device))

    def _call(self, name, args, stream):
        status = getattr(self.lib, name)(*args, stream)
        if status:
            raise PagedKVError(name, status)

    def write(self, stream=None):
        self._call(self._write, self.write_args, _stream(stream, self._write_device))

    def slot_map_and_write(self, stream=None):
        self._call(self._mapped_write, self.mapped_write_args,
                   _stream(stream, self._write_device))

    def attend(self, stream=None):
        self._call(self._attend, self.attn_args, _stream(stream, self._device))

    def run(self, stream=None):
        st = _stream(stream, self._device)
        if self.write_in_attention:
            self._call(self._attend_write, self.attn_write_args, st)
            return
        if self.fused_write:
            self._call(self._mapped_write, self.mapped_write_args, st)
        else:
            self._call("pkv_slot_mapping", self.slot_args, st)
            self._call(self._write, self.write_args, st)
        self._call(self._attend, self.attn_args, st)
