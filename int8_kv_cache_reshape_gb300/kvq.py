"""ctypes binding of libkvq.so (include/kvq.h) -- argument marshalling only.

Every function here turns tensors into pointers and sizes and calls the C
ABI of the same name; all computation runs in the library's CUDA kernels.
Importing this module loads the library and raises if it was not built
(``python -m int8_kv_cache_reshape_gb300.build`` or ``__graft_entry__.build()``):
there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# KVQ_LIBRARY selects another build of the library (the bounds-checked
# libkvq_checked.so); default libkvq.so next to this file.
LIB_PATH = os.environ.get("KVQ_LIBRARY") or os.path.join(_HERE, "libkvq.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "kvq.h")

OK = 0
E_INVALID_ARG, E_UNSUPPORTED, E_SCHED_MISMATCH = -1, -2, -3
E_WORKSPACE_TOO_SMALL, E_CUDA, E_NO_MEMORY, E_TIMEOUT = -4, -5, -6, -7

DTYPES = {"auto": 0, "fp8_e4m3": 1, "fp8_e5m2": 2, "int8_per_token_head": 3,
          "fp8_per_token_head": 4, "fp8_e5m2_per_token_head": 5, "int4_per_token_head": 6}


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{os.path.basename(LIB_PATH)} is not built ({LIB_PATH}); run "
                      "int8_kv_cache_reshape_gb300.build.build() first")

lib = ctypes.CDLL(LIB_PATH)


class SchedInfo(ctypes.Structure):
    _fields_ = [("num_req", ctypes.c_int), ("heads_q", ctypes.c_int),
                ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("kv_elem_bytes", ctypes.c_int),
                ("row_bytes", ctypes.c_int), ("causal", ctypes.c_int),
                ("window", ctypes.c_int),
                ("num_tiles", ctypes.c_int64),
                ("num_pieces", ctypes.c_int64),
                ("num_merge_items", ctypes.c_int64),
                ("num_chunks", ctypes.c_int64),
                ("num_decode_warps", ctypes.c_int64),
                ("max_splits", ctypes.c_int64),
                ("total_query_tokens", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_size_t),
                ("decode_smem_bytes", ctypes.c_size_t),
                ("decode_chunk_bytes", ctypes.c_size_t),
                ("num_prefill_tiles", ctypes.c_int64),
                ("prefill_smem_bytes", ctypes.c_size_t),
                ("num_kernel_launches", ctypes.c_int64),
                ("prefill_cta_group", ctypes.c_int64)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


_c = ctypes
_p = ctypes.c_void_p
lib.kvq_status_string.restype = _c.c_char_p
lib.kvq_status_string.argtypes = [_c.c_int]
lib.kvq_parse_kv_cache_dtype.restype = _c.c_int
lib.kvq_parse_kv_cache_dtype.argtypes = [_c.c_char_p, _c.POINTER(_c.c_int)]
lib.kvq_cache_row_bytes.restype = _c.c_int
lib.kvq_cache_row_bytes.argtypes = [_c.c_int, _c.c_int, _c.POINTER(_c.c_size_t)]
lib.kvq_reshape_and_cache.restype = _c.c_int
lib.kvq_reshape_and_cache.argtypes = [
    _p, _p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int, _p, _p,
    _c.c_int64, _c.c_int, _p, _c.c_int, _c.c_float, _c.c_float, _p]
lib.kvq_gather_cache.restype = _c.c_int
lib.kvq_gather_cache.argtypes = [
    _p, _p, _c.c_int64, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_float, _c.c_float, _p,
    _c.c_int64, _c.c_int, _p, _p, _c.c_int64, _c.c_int64, _p]
lib.kvq_build_block_tables.restype = _c.c_int
lib.kvq_build_block_tables.argtypes = [
    _c.c_int, _p, _p, _p, _c.c_int64, _p, _p, _c.c_int, _p, _c.c_int64, _c.c_int, _c.c_int64,
    _p, _p, _p]
lib.kvq_get_scheduler_metadata.restype = _c.c_int
lib.kvq_get_scheduler_metadata.argtypes = [
    _c.c_int, _c.c_int, _c.c_int, _c.c_int, _p, _p, _c.c_int, _c.c_int,
    _c.c_int, _c.POINTER(_p), _c.POINTER(_c.c_size_t)]
lib.kvq_attention_with_kv_cache.restype = _c.c_int
lib.kvq_attention_with_kv_cache.argtypes = [
    _p, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _p, _p, _p, _p, _p, _p,
    _c.c_int, _c.c_int, _c.c_int64, _c.c_float, _c.c_int, _c.c_int,
    _c.c_float, _p, _p, _c.c_float, _c.c_float, _p, _p, _c.c_size_t, _p]
lib.kvq_attention_with_kv_cache_static_scratch.restype = _c.c_int
lib.kvq_attention_with_kv_cache_static_scratch.argtypes = [
    _p, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _p, _p, _p, _p, _p, _p,
    _c.c_int, _c.c_int, _c.c_int64, _c.c_float, _c.c_int, _c.c_int,
    _c.c_float, _p, _p, _c.c_float, _c.c_float, _p, _p]
STATIC_SCRATCH_BYTES = 16 << 20
lib.kvq_decode_step.restype = _c.c_int
lib.kvq_decode_step.argtypes = [
    _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _p, _p, _c.c_int64, _c.c_int64,
    _c.c_int64, _p, _p, _p, _c.c_int64, _c.c_int, _p, _p, _p, _p, _c.c_int, _c.c_int,
    _c.c_float, _c.c_int, _c.c_float, _p, _p, _c.c_float, _c.c_float, _p, _p, _c.c_size_t, _p]
lib.kvq_decode_step_host_io.restype = _c.c_int
lib.kvq_decode_step_host_io.argtypes = [_p, _p, _c.c_size_t, _p, _c.c_size_t] + lib.kvq_decode_step.argtypes
lib.kvq_decode_step_graph_create.restype = _c.c_int
lib.kvq_decode_step_graph_create.argtypes = ([_p, _p, _c.c_size_t, _p, _c.c_size_t]
                                             + lib.kvq_decode_step.argtypes[:-1]
                                             + [_c.POINTER(_p)])
lib.kvq_decode_step_graph_launch.restype = _c.c_int
lib.kvq_decode_step_graph_launch.argtypes = [_p, _p]
lib.kvq_decode_step_graph_destroy.restype = None
lib.kvq_decode_step_graph_destroy.argtypes = [_p]
lib.kvq_decode_step_workspace_size.restype = _c.c_int
lib.kvq_decode_step_workspace_size.argtypes = [
    _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.POINTER(_c.c_size_t)]
lib.kvq_decode_step_check.restype = _c.c_int
lib.kvq_decode_step_check.argtypes = [_p]
lib.kvq_sched_destroy.restype = None
lib.kvq_sched_destroy.argtypes = [_p]
lib.kvq_sched_check_device.restype = _c.c_int
lib.kvq_sched_check_device.argtypes = [_p]
lib.kvq_sched_get_info.restype = _c.c_int
lib.kvq_sched_get_info.argtypes = [_p, _c.POINTER(SchedInfo)]


class PlanSizes(ctypes.Structure):
    _fields_ = [("num_pieces", ctypes.c_int64), ("num_merges", ctypes.c_int64),
                ("num_prefill_tiles", ctypes.c_int64), ("num_chunks", ctypes.c_int64 * 2),
                ("num_warps", ctypes.c_int32 * 2), ("lockstep", ctypes.c_int32 * 2)]


# numpy layouts of kvq_plan_piece_t, kvq_plan_merge_t, kvq_plan_prefill_tile_t
PLAN_PIECE = np.dtype([(n, np.int32) for n in (
    "launch", "req", "kv_head", "row0", "nrows", "part", "merge", "key_lo", "key_hi", "flat0",
    "chunk0", "nchunks")])
PLAN_MERGE = np.dtype([(n, np.int32) for n in ("req", "kv_head", "row0", "nrows", "part",
                                                "nsplits")])
PLAN_PREFILL = np.dtype([(n, np.int32) for n in ("req", "kv_head", "row0", "nrows", "key_lo",
                                                  "key_hi")])
lib.kvq_sched_get_plan_sizes.restype = _c.c_int
lib.kvq_sched_get_plan_sizes.argtypes = [_p, _c.POINTER(PlanSizes)]
lib.kvq_sched_export_plan.restype = _c.c_int
lib.kvq_sched_export_plan.argtypes = [_p, _p, _c.c_int64, _p, _c.c_int64, _p, _c.c_int64, _p,
                                      _c.c_int64]


def declared_functions() -> list:
    """Names of the functions include/kvq.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kvq_\w+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib.kvq_status_string(int(status)).decode()


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise KvqError(rc, what)


def _ptr(t):
    return None if t is None else _p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return _p(getattr(stream, "cuda_stream", stream))


def parse_kv_cache_dtype(s) -> int:
    out = _c.c_int()
    _check(lib.kvq_parse_kv_cache_dtype(None if s is None else s.encode(), _c.byref(out)),
           "kvq_parse_kv_cache_dtype")
    return out.value


def cache_row_bytes(kv_cache_dtype, head_dim: int) -> int:
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    out = _c.c_size_t()
    _check(lib.kvq_cache_row_bytes(dt, head_dim, _c.byref(out)), "kvq_cache_row_bytes")
    return out.value


@functools.lru_cache(maxsize=None)
def _row_bytes(dt: int, head_dim: int) -> int:
    """cache_row_bytes, looked up once."""
    return cache_row_bytes(dt, head_dim)


def _flat(name, t, dtype, least=0):
    """t as the library reads it: contiguous, of the dtype, of `least` elements or more."""
    if t.dtype != dtype or not t.is_contiguous() or t.numel() < least:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {least} elements")


def _reshape_and_cache_args(key, value, key_cache, value_cache, slot_mapping, kv_cache_dtype,
                            k_scale, v_scale, stream):
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    T, H, D = key.shape
    return (_ptr(key), _ptr(value), T, key.stride(0), value.stride(0), H, D, _ptr(key_cache),
            _ptr(value_cache), key_cache.shape[0], key_cache.shape[1], _ptr(slot_mapping), dt,
            float(k_scale), float(v_scale), _stream(stream))


def reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, kv_cache_dtype,
                      k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """key/value: bf16 [T, Hkv, D] (token stride may exceed Hkv*D);
    caches: uint8 [NB, B, Hkv, row]; slot_mapping: int64 [T]."""
    _check(lib.kvq_reshape_and_cache(*_reshape_and_cache_args(
        key, value, key_cache, value_cache, slot_mapping, kv_cache_dtype, k_scale, v_scale,
        stream)), "kvq_reshape_and_cache")


class Prepared:
    """One C-ABI call with its arguments marshalled once (pointers, sizes,
    the stream), for a serving loop that calls it every step on the same
    buffers: calling the object only crosses into the library.  The tensors
    behind the pointers must stay alive (and in place) while it is used."""

    def __init__(self, fn, args, what: str):
        self.fn = fn
        self.args = tuple(args)
        self.what = what

    def __call__(self) -> None:
        _check(self.fn(*self.args), self.what)


def _marshalled(fn, args):
    """The arguments as ctypes values of fn's declared types, converted once."""
    return [a if isinstance(a, (t, type(None))) else t(a) for t, a in zip(fn.argtypes, args)]


def prepare_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, kv_cache_dtype,
                              k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> Prepared:
    """reshape_and_cache with its arguments marshalled once (see Prepared)."""
    return Prepared(lib.kvq_reshape_and_cache, _marshalled(
        lib.kvq_reshape_and_cache, _reshape_and_cache_args(
            key, value, key_cache, value_cache, slot_mapping, kv_cache_dtype, k_scale, v_scale,
            stream)), "kvq_reshape_and_cache")


def _gather_cache_args(key_cache, value_cache, slot_mapping, key_out, value_out, kv_cache_dtype,
                       k_scale, v_scale, stream):
    import torch
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    T, H, D = key_out.shape
    if key_out.dtype != value_out.dtype or key_out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("key_out and value_out must both be bfloat16 or both float32")
    if tuple(value_out.shape) != (T, H, D) or tuple(slot_mapping.shape) != (T,):
        raise ValueError("key_out, value_out and slot_mapping must agree on their rows")
    _flat("slot_mapping", slot_mapping, torch.int64)
    for t in (key_out, value_out):
        if T > 0 and (t.stride(2) != 1 or (H > 1 and t.stride(1) != D)):
            raise ValueError("the heads and dims of key_out and value_out must be contiguous")
    # The library reads rows of H heads of D dims at the slots of the pool.
    row = _row_bytes(dt, D)
    for t in (key_cache, value_cache):
        if t.dim() != 4 or t.shape[2] != H or t.shape[3] * t.element_size() != row or not t.is_contiguous():
            raise ValueError(f"the caches must be contiguous [num_blocks, block_size, {H}, {row} bytes]")
    if key_cache.shape != value_cache.shape:
        raise ValueError("key_cache and value_cache must have one shape")
    return (_ptr(key_cache), _ptr(value_cache), key_cache.shape[0], key_cache.shape[1], H, D, dt,
            float(k_scale), float(v_scale), _ptr(slot_mapping), T,
            int(key_out.dtype == torch.float32), _ptr(key_out), _ptr(value_out),
            key_out.stride(0), value_out.stride(0), _stream(stream))


def gather_cache(key_cache, value_cache, slot_mapping, key_out, value_out, kv_cache_dtype,
                 k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Cache rows read back as values: caches uint8 [NB, B, Hkv, row];
    slot_mapping int64 [T]; key_out / value_out bf16 or float32 [T, Hkv, D]
    (token stride may exceed Hkv*D)."""
    _check(lib.kvq_gather_cache(*_gather_cache_args(
        key_cache, value_cache, slot_mapping, key_out, value_out, kv_cache_dtype, k_scale,
        v_scale, stream)), "kvq_gather_cache")


def prepare_gather_cache(key_cache, value_cache, slot_mapping, key_out, value_out, kv_cache_dtype,
                         k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> Prepared:
    """gather_cache with its arguments marshalled once (see Prepared)."""
    return Prepared(lib.kvq_gather_cache, _marshalled(lib.kvq_gather_cache, _gather_cache_args(
        key_cache, value_cache, slot_mapping, key_out, value_out, kv_cache_dtype, k_scale,
        v_scale, stream)), "kvq_gather_cache")


def _build_block_tables_args(query_start_loc, seq_lens, free_blocks, free_count, block_table,
                             slot_mapping, block_size, num_blocks, free_count_out, status, stream):
    import torch
    R = seq_lens.numel()
    for name, t, dtype, least in (
            ("query_start_loc", query_start_loc, torch.int32, R + 1), ("seq_lens", seq_lens, torch.int32, 0),
            ("free_blocks", free_blocks, torch.int32, 0), ("free_count", free_count, torch.int32, 1),
            ("slot_mapping", slot_mapping, torch.int64, 0),
            ("free_count_out", free_count_out, torch.int32, 1), ("status", status, torch.int32, 4)):
        _flat(name, t, dtype, least)
    if query_start_loc.numel() != R + 1 or block_table.dim() != 2 or block_table.shape[0] < R:
        raise ValueError("query_start_loc, seq_lens and block_table must agree on their requests")
    # The library's one stride is both the rows' pitch and their width, so a
    # view of some columns (a pitch beyond its width) would let a request
    # store into columns that the caller did not hand over.  (One row has no
    # pitch.)
    width = block_table.shape[1]
    if block_table.dtype != torch.int32 or (width > 1 and block_table.stride(1) != 1) or (
            R > 1 and block_table.stride(0) != width):
        raise ValueError("block_table must be int32 rows side by side (not a view of some columns)")
    return (R, _ptr(query_start_loc), _ptr(seq_lens), _ptr(free_blocks), free_blocks.numel(),
            _ptr(free_count), _ptr(block_table), width, _ptr(slot_mapping),
            slot_mapping.numel(), int(block_size), int(num_blocks), _ptr(free_count_out),
            _ptr(status), _stream(stream))


def build_block_tables(query_start_loc, seq_lens, free_blocks, free_count, block_table,
                       slot_mapping, block_size: int, num_blocks: int, free_count_out, status,
                       stream=None) -> None:
    """Block tables and slot mapping of a step on the device: query_start_loc
    int32 [R + 1], seq_lens int32 [R], free_blocks int32 (a stack of
    free_count int32 [1] ids), block_table int32 [R, width] (rows side by
    side; entries of new blocks are stored), slot_mapping int64 (padded
    entries get -1),
    free_count_out int32 [1] (may be free_count), status int32 [4],
    zero-filled before its first use."""
    _check(lib.kvq_build_block_tables(*_build_block_tables_args(
        query_start_loc, seq_lens, free_blocks, free_count, block_table, slot_mapping, block_size,
        num_blocks, free_count_out, status, stream)), "kvq_build_block_tables")


def prepare_build_block_tables(query_start_loc, seq_lens, free_blocks, free_count, block_table,
                               slot_mapping, block_size: int, num_blocks: int, free_count_out,
                               status, stream=None) -> Prepared:
    """build_block_tables with its arguments marshalled once (see Prepared)."""
    return Prepared(lib.kvq_build_block_tables, _marshalled(
        lib.kvq_build_block_tables, _build_block_tables_args(
            query_start_loc, seq_lens, free_blocks, free_count, block_table, slot_mapping,
            block_size, num_blocks, free_count_out, status, stream)), "kvq_build_block_tables")


class Sched:
    """Owns one kvq_sched_t (freed on close / garbage collection)."""

    def __init__(self, handle, workspace_bytes: int):
        self.handle = handle
        self.workspace_bytes = workspace_bytes

    def info(self) -> dict:
        inf = SchedInfo()
        _check(lib.kvq_sched_get_info(self.handle, _c.byref(inf)), "kvq_sched_get_info")
        return inf.as_dict()

    def plan(self) -> dict:
        """The schedule's plan as numpy arrays (kvq_sched_export_plan)."""
        sz = PlanSizes()
        _check(lib.kvq_sched_get_plan_sizes(self.handle, _c.byref(sz)), "kvq_sched_get_plan_sizes")
        pieces = np.zeros(sz.num_pieces, PLAN_PIECE)
        warps = np.zeros(sz.num_warps[0] + sz.num_warps[1], np.int32)
        merges = np.zeros(sz.num_merges, PLAN_MERGE)
        tiles = np.zeros(sz.num_prefill_tiles, PLAN_PREFILL)
        _check(lib.kvq_sched_export_plan(
            self.handle, pieces.ctypes.data, pieces.size, warps.ctypes.data, warps.size,
            merges.ctypes.data, merges.size, tiles.ctypes.data, tiles.size),
            "kvq_sched_export_plan")
        return {"pieces": pieces, "warp_first_piece": warps, "merges": merges,
                "prefill_tiles": tiles, "num_chunks": list(sz.num_chunks),
                "num_warps": list(sz.num_warps), "lockstep": list(sz.lockstep)}

    def check_device(self) -> None:
        """Raise KvqError(E_TIMEOUT) if a kernel run with this schedule gave
        up a bounded wait; synchronizes the device."""
        _check(lib.kvq_sched_check_device(self.handle), "kvq_sched_check_device")

    def close(self):
        if self.handle is not None:
            lib.kvq_sched_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


def get_scheduler_metadata(num_req: int, heads_q: int, heads_kv: int, head_dim: int,
                           seq_lens, query_start_loc, causal: bool, window: int,
                           kv_cache_dtype) -> Sched:
    """seq_lens / query_start_loc: host int32 tensors or arrays."""
    import numpy as np
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    sl = np.ascontiguousarray(np.asarray(seq_lens), dtype=np.int32)
    qsl = np.ascontiguousarray(np.asarray(query_start_loc), dtype=np.int32)
    h = _p()
    ws = _c.c_size_t()
    _check(lib.kvq_get_scheduler_metadata(
        num_req, heads_q, heads_kv, head_dim, _p(sl.ctypes.data), _p(qsl.ctypes.data),
        int(bool(causal)), int(window), dt, _c.byref(h), _c.byref(ws)),
        "kvq_get_scheduler_metadata")
    return Sched(h, ws.value)


def _attention_args(sched, q, key_cache, value_cache, query_start_loc, seq_lens, block_table,
                    sm_scale, causal, window, soft_cap, k_scale, v_scale, out, workspace,
                    kv_cache_dtype, heads_kv, stream, num_blocks, alibi_slopes, sinks):
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    _, Hq, D = q.shape
    nb = key_cache.shape[0] if num_blocks is None else num_blocks
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return (sched.handle, Hq, heads_kv, D, dt, _ptr(q), _ptr(key_cache), _ptr(value_cache),
            _ptr(query_start_loc), _ptr(seq_lens), _ptr(block_table), block_table.stride(0),
            key_cache.shape[1], nb, float(sm_scale), int(bool(causal)), int(window),
            float(soft_cap), _ptr(alibi_slopes), _ptr(sinks), float(k_scale), float(v_scale),
            _ptr(out), _ptr(workspace), ws_bytes, _stream(stream))


def attention_with_kv_cache(sched: Sched, q, key_cache, value_cache, query_start_loc,
                            seq_lens, block_table, sm_scale: float, causal: bool,
                            window: int, soft_cap: float, k_scale: float, v_scale: float,
                            out, workspace, kv_cache_dtype, heads_kv: int, stream=None,
                            num_blocks=None, alibi_slopes=None, sinks=None) -> None:
    """q / out: bf16 [sum Q, Hq, D]; caches uint8 [NB, B, Hkv, row];
    block_table int32 [R, max_blocks]; query_start_loc / seq_lens device
    int32; workspace: a uint8 device tensor of >= sched.workspace_bytes;
    alibi_slopes / sinks: device float32 [Hq] or None."""
    _check(lib.kvq_attention_with_kv_cache(*_attention_args(
        sched, q, key_cache, value_cache, query_start_loc, seq_lens, block_table, sm_scale,
        causal, window, soft_cap, k_scale, v_scale, out, workspace, kv_cache_dtype, heads_kv,
        stream, num_blocks, alibi_slopes, sinks)), "kvq_attention_with_kv_cache")


def prepare_attention_with_kv_cache(sched: Sched, q, key_cache, value_cache, query_start_loc,
                                    seq_lens, block_table, sm_scale: float, causal: bool,
                                    window: int, soft_cap: float, k_scale: float, v_scale: float,
                                    out, workspace, kv_cache_dtype, heads_kv: int, stream=None,
                                    num_blocks=None, alibi_slopes=None, sinks=None) -> Prepared:
    """attention_with_kv_cache with its arguments marshalled once (see
    Prepared): the layers of a step, or steps replayed with one schedule,
    which must stay open too."""
    return Prepared(lib.kvq_attention_with_kv_cache, _marshalled(
        lib.kvq_attention_with_kv_cache, _attention_args(
            sched, q, key_cache, value_cache, query_start_loc, seq_lens, block_table, sm_scale,
            causal, window, soft_cap, k_scale, v_scale, out, workspace, kv_cache_dtype, heads_kv,
            stream, num_blocks, alibi_slopes, sinks)), "kvq_attention_with_kv_cache")


def attention_with_kv_cache_static_scratch(sched: Sched, q, key_cache, value_cache,
                                           query_start_loc, seq_lens, block_table,
                                           sm_scale: float, causal: bool, window: int,
                                           soft_cap: float, k_scale: float, v_scale: float,
                                           out, kv_cache_dtype, heads_kv: int, stream=None,
                                           num_blocks=None, alibi_slopes=None,
                                           sinks=None) -> None:
    """attention_with_kv_cache without a workspace argument: the library's
    fixed device scratch (STATIC_SCRATCH_BYTES) holds the split partials.
    For callers that cannot allocate device memory; calls must not overlap
    on the GPU."""
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    _, Hq, D = q.shape
    nb = key_cache.shape[0] if num_blocks is None else num_blocks
    _check(lib.kvq_attention_with_kv_cache_static_scratch(
        sched.handle, Hq, heads_kv, D, dt, _ptr(q), _ptr(key_cache), _ptr(value_cache),
        _ptr(query_start_loc), _ptr(seq_lens), _ptr(block_table), block_table.stride(0),
        key_cache.shape[1], nb, float(sm_scale), int(bool(causal)), int(window),
        float(soft_cap), _ptr(alibi_slopes), _ptr(sinks), float(k_scale), float(v_scale),
        _ptr(out), _stream(stream)), "kvq_attention_with_kv_cache_static_scratch")


def decode_step_workspace_size(num_req: int, heads_q: int, heads_kv: int, head_dim: int,
                               kv_cache_dtype, max_query_len: int = 1,
                               use_alibi: bool = False) -> int:
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    out = _c.c_size_t()
    _check(lib.kvq_decode_step_workspace_size(num_req, heads_q, heads_kv, head_dim, dt,
                                              max_query_len, int(bool(use_alibi)),
                                              _c.byref(out)), "kvq_decode_step_workspace_size")
    return out.value


def _decode_step_args(key, value, slot_mapping, key_cache, value_cache, q, query_start_loc,
                      seq_lens, block_table, max_query_len, sm_scale, window, soft_cap, k_scale,
                      v_scale, out, workspace, kv_cache_dtype, heads_kv, alibi_slopes, sinks,
                      stream, num_blocks):
    dt = parse_kv_cache_dtype(kv_cache_dtype) if isinstance(kv_cache_dtype, str) else kv_cache_dtype
    _, Hq, D = q.shape
    T = key.shape[0]
    nb = key_cache.shape[0] if num_blocks is None else num_blocks
    return (_c.c_int(seq_lens.shape[0]), _c.c_int(Hq), _c.c_int(heads_kv), _c.c_int(D),
            _c.c_int(dt), _ptr(key), _ptr(value), _c.c_int64(T), _c.c_int64(key.stride(0)),
            _c.c_int64(value.stride(0)), _ptr(slot_mapping), _ptr(key_cache), _ptr(value_cache),
            _c.c_int64(nb), _c.c_int(key_cache.shape[1]), _ptr(q), _ptr(query_start_loc),
            _ptr(seq_lens), _ptr(block_table), _c.c_int(block_table.stride(0)),
            _c.c_int(int(max_query_len)), _c.c_float(sm_scale), _c.c_int(int(window)),
            _c.c_float(soft_cap), _ptr(alibi_slopes), _ptr(sinks), _c.c_float(k_scale),
            _c.c_float(v_scale), _ptr(out), _ptr(workspace),
            _c.c_size_t(workspace.numel() * workspace.element_size()), _stream(stream))


def decode_step(key, value, slot_mapping, key_cache, value_cache, q, query_start_loc, seq_lens,
                block_table, max_query_len: int, sm_scale: float, window: int, soft_cap: float,
                k_scale: float, v_scale: float, out, workspace, kv_cache_dtype, heads_kv: int,
                alibi_slopes=None, sinks=None, stream=None, num_blocks=None) -> None:
    """kvq_decode_step: the new rows key/value bf16 [T, Hkv, D] with their
    slot_mapping int64 [T]; q / out bf16 [sum Q, Hq, D]; query_start_loc,
    seq_lens int32 device; workspace: a zero-filled uint8 device tensor of
    >= decode_step_workspace_size(...) bytes."""
    _check(lib.kvq_decode_step(*_decode_step_args(
        key, value, slot_mapping, key_cache, value_cache, q, query_start_loc, seq_lens,
        block_table, max_query_len, sm_scale, window, soft_cap, k_scale, v_scale, out, workspace,
        kv_cache_dtype, heads_kv, alibi_slopes, sinks, stream, num_blocks)), "kvq_decode_step")


def prepare_decode_step(key, value, slot_mapping, key_cache, value_cache, q, query_start_loc,
                        seq_lens, block_table, max_query_len: int, sm_scale: float, window: int,
                        soft_cap: float, k_scale: float, v_scale: float, out, workspace,
                        kv_cache_dtype, heads_kv: int, alibi_slopes=None, sinks=None,
                        stream=None, num_blocks=None) -> Prepared:
    """decode_step with its arguments marshalled once (see Prepared)."""
    return Prepared(lib.kvq_decode_step, _decode_step_args(
        key, value, slot_mapping, key_cache, value_cache, q, query_start_loc, seq_lens,
        block_table, max_query_len, sm_scale, window, soft_cap, k_scale, v_scale, out, workspace,
        kv_cache_dtype, heads_kv, alibi_slopes, sinks, stream, num_blocks), "kvq_decode_step")


def _host_io_args(host_in, dev_in, host_out, out_bytes):
    in_bytes = host_in.numel() * host_in.element_size()
    if dev_in.numel() * dev_in.element_size() < in_bytes:
        raise ValueError("dev_in is smaller than host_in")
    if out_bytes > host_out.numel() * host_out.element_size():
        raise ValueError("out_bytes exceeds host_out")
    return (_ptr(host_in), _ptr(dev_in), _c.c_size_t(in_bytes), _ptr(host_out),
            _c.c_size_t(int(out_bytes)))


def prepare_decode_step_host_io(host_in, dev_in, host_out, out_bytes: int, key, value,
                                slot_mapping, key_cache, value_cache, q, query_start_loc,
                                seq_lens, block_table, max_query_len: int, sm_scale: float,
                                window: int, soft_cap: float, k_scale: float, v_scale: float,
                                out, workspace, kv_cache_dtype, heads_kv: int, alibi_slopes=None,
                                sinks=None, stream=None, num_blocks=None) -> Prepared:
    """kvq_decode_step_host_io, marshalled once (see Prepared): each call
    copies host_in (a pinned uint8 tensor) to dev_in, runs the decode step
    (whose device tensors may be views of dev_in), copies out_bytes of out
    to host_out (pinned) and waits for the stream.  out None: the step
    writes its output straight into host_out (out_bytes ignored)."""
    return Prepared(lib.kvq_decode_step_host_io, _host_io_args(host_in, dev_in, host_out, out_bytes)
                    + _decode_step_args(key, value, slot_mapping, key_cache, value_cache, q,
                                        query_start_loc, seq_lens, block_table, max_query_len,
                                        sm_scale, window, soft_cap, k_scale, v_scale, out,
                                        workspace, kv_cache_dtype, heads_kv, alibi_slopes, sinks,
                                        stream, num_blocks), "kvq_decode_step_host_io")


class DecodeStepGraph:
    """A host-buffer decode step captured once in a CUDA graph
    (kvq_decode_step_graph_create); calling it replays the step on the
    stream it was made for and waits (kvq_decode_step_graph_launch).  The
    buffers behind it must stay alive, in place, until close()."""

    def __init__(self, handle, stream):
        self._h = handle
        self._stream = stream
        self._launch = lib.kvq_decode_step_graph_launch

    def __call__(self) -> None:
        _check(self._launch(self._h, self._stream), "kvq_decode_step_graph_launch")

    def close(self) -> None:
        if self._h:
            lib.kvq_decode_step_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def decode_step_graph(host_in, dev_in, host_out, out_bytes: int, key, value, slot_mapping,
                      key_cache, value_cache, q, query_start_loc, seq_lens, block_table,
                      max_query_len: int, sm_scale: float, window: int, soft_cap: float,
                      k_scale: float, v_scale: float, out, workspace, kv_cache_dtype,
                      heads_kv: int, alibi_slopes=None, sinks=None, stream=None,
                      num_blocks=None) -> DecodeStepGraph:
    """kvq_decode_step_graph_create with the arguments of
    prepare_decode_step_host_io; host_in must be pinned (the fused kernel
    stages it).  Rewrite host_in between calls of the returned object."""
    args = (_host_io_args(host_in, dev_in, host_out, out_bytes)
            + _decode_step_args(key, value, slot_mapping, key_cache, value_cache, q,
                                query_start_loc, seq_lens, block_table, max_query_len, sm_scale,
                                window, soft_cap, k_scale, v_scale, out, workspace,
                                kv_cache_dtype, heads_kv, alibi_slopes, sinks, stream,
                                num_blocks))
    h = _p()
    _check(lib.kvq_decode_step_graph_create(*args[:-1], _c.byref(h)), "kvq_decode_step_graph_create")
    return DecodeStepGraph(h, args[-1])


def decode_step_check(workspace) -> None:
    """Raise KvqError if a decode_step run with this workspace flagged an
    error (synchronises the device)."""
    _check(lib.kvq_decode_step_check(_ptr(workspace)), "kvq_decode_step_check")
