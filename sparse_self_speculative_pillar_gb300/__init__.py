"""GB300 (sm_103a) PillarAttn unified step: thin Python binding over the C ABI.

Every step of the path runs in the CUDA library built from ``csrc/``; this
module only marshals arguments (torch tensors or raw device pointers) into
the ``extern "C"`` entry points declared in ``include/pillar.h`` and turns
non-zero status codes into exceptions.  There is no fallback: if the
library is missing or cannot be loaded, every call raises.

Entry points (same names as the C ABI):
  pillar_attn_workspace_bytes(shape)
  pillar_attn_unified(shape, q, k_pool, v_pool, slot_table, req_mode, req_len,
                      sparse_idx, sparse_cnt, out, verify_logits, verify_lse,
                      workspace, stream=None)
  pillar_topk_workspace_bytes(shape, V)
  pillar_topk_select(shape, V, verify_logits, verify_lse, req_len, group_map, K,
                     next_idx, next_cnt, workspace, stream=None)
  pillar_get_error(workspace, stream=None)
  pillar_status_string(status)
  pillar_attn_unified_slotted(shape, ..., sparse_slot, out, ...)   (draft lists with their slots)
  pillar_attn_plan(shape, req_mode, req_len, sparse_cnt, workspace, stream=None)
  pillar_attn_run(shape, q, k_pool, v_pool, slot_table, sparse_idx, out, verify_logits, verify_lse,
                  workspace, sparse_slot=None, stream=None)  (one plan, several runs)
  pillar_draft_lists(shape, V, next_idx, next_cnt, group_map, verify_len, req_len, slot_table,
                     sparse_idx, sparse_cnt, sparse_slot=None, device_flags=None, stream=None)
  pillar_topk_select_noalloc(shape, V, ..., device_flags=None, stream=None)
  pillar_kv_append(shape, k_new, v_new, slots, k_pool, v_pool, device_flags=None, stream=None)
  pillar_kv_offload(shape, k_pool, v_pool, slots, host_k, host_v, device_flags=None, stream=None)
  pillar_kv_reload(shape, host_k, host_v, slots, k_pool, v_pool, device_flags=None, stream=None)
  pillar_buckets_init(k), pillar_buckets_admit(pb), pillar_buckets_retire(pb, bucket),
  pillar_buckets_step(pb, buckets, step)    (host-side phase buckets)
  pillar_offload_init(capacity, chunk), pillar_offload_reserve(f, n, new_request),
  pillar_offload_release(f, n), pillar_offload_evict(f, req, len),
  pillar_offload_reload(f, max_out)         (host-side FIFO of offloaded KV chunks)
  pillar_block_map_workspace_bytes(shape)
  pillar_block_map(shape, req_len, prev_len, block_table, free_ring, free_state, granted_len, kv_off, slot_table,
                   new_off, new_slots, workspace, stream=None)   (block tables and slot maps from lengths)
  pillar_kv8_append(shape, k_new, v_new, req_len, new_off, block_table, k8_pool, v8_pool, k_scale, v_scale,
                    device_flags=None, stream=None)              (new rows into the 8-bit cache)
  pillar_attn_kv8(shape, q, k8_pool, v8_pool, k_scale, v_scale, block_table, req_mode, req_len, sparse_idx, sparse_cnt,
                  out, verify_logits, verify_lse, workspace, stream=None)   (the unified step over the 8-bit cache)
  pillar_attn_run_kv8(shape, q, k8_pool, v8_pool, k_scale, v_scale, block_table, sparse_idx, out, verify_logits,
                      verify_lse, workspace, stream=None)        (the same on a plan of pillar_attn_plan)
  pillar_kv8_read(shape, k8_pool, v8_pool, k_scale, v_scale, block_table, first, out_off, k_out, v_out,
                  device_flags=None, stream=None)                (positions of the 8-bit cache as bf16 rows)
  pillar_kv4_append(...), pillar_kv4_read(...), pillar_attn_kv4(...), pillar_attn_run_kv4(...)
                                                                 (the same four over the 4-bit cache)
  pillar_prompt_attn_workspace_bytes(shape, n)
  pillar_prompt_attn(shape, q, k, v, seq_off, out, lse, workspace, stream=None)   (causal attention over packed prompts)
"""
from __future__ import annotations

import ctypes
import os

from . import _build

__all__ = [
    "PillarShape", "make_shape", "PillarError", "load", "library_path", "build",
    "pillar_attn_workspace_bytes", "pillar_attn_unified", "pillar_attn_unified_slotted", "pillar_draft_lists",
    "pillar_attn_plan", "pillar_attn_run",
    "pillar_topk_workspace_bytes", "pillar_topk_select", "pillar_topk_select_noalloc", "pillar_get_error", "pillar_status_string",
    "FLAG_INDEX", "FLAG_SLOT", "FLAG_REQUEST", "FLAG_COUNT", "FLAG_TIMEOUT", "FLAG_TOPK",
    "SCHEDULE_UNIFIED", "SCHEDULE_DRAFT_ONLY", "SCHEDULE_VERIFY_ONLY", "SCHEDULE_UNIFORM_ROWS", "SCHEDULE_NAIVE_JOINT",
    "pillar_kv_append", "PillarBuckets", "pillar_buckets_init", "pillar_buckets_admit", "pillar_buckets_retire", "pillar_buckets_step",
    "pillar_kv_offload", "pillar_kv_reload", "PillarOffloadFifo", "pillar_offload_init", "pillar_offload_reserve",
    "pillar_offload_release", "pillar_offload_evict", "pillar_offload_reload",
    "pillar_block_map_workspace_bytes", "pillar_block_map", "pillar_kv8_append",
    "pillar_attn_kv8", "pillar_attn_run_kv8", "pillar_prompt_attn_workspace_bytes", "pillar_prompt_attn",
    "pillar_kv8_read", "pillar_kv4_append", "pillar_kv4_read", "pillar_attn_kv4", "pillar_attn_run_kv4",
    "FLAG_BLOCK", "FLAG_VALUE", "KV_BLOCK", "KV4_GROUP",
]

FLAG_INDEX, FLAG_SLOT, FLAG_REQUEST, FLAG_COUNT, FLAG_TIMEOUT, FLAG_TOPK = 1, 2, 4, 8, 16, 32
FLAG_BLOCK, FLAG_VALUE = 64, 128
KV_BLOCK = 16  # PILLAR_KV_BLOCK: tokens of a cache block
KV4_GROUP = 16  # PILLAR_KV4_GROUP: values of a row that share a scale byte in the 4-bit cache
# values of PillarShape.schedule (PILLAR_SCHEDULE_* in the header)
SCHEDULE_UNIFIED, SCHEDULE_DRAFT_ONLY, SCHEDULE_VERIFY_ONLY, SCHEDULE_UNIFORM_ROWS, SCHEDULE_NAIVE_JOINT = 0, 1, 2, 3, 4
EXPORTED = ("pillar_attn_workspace_bytes", "pillar_attn_unified", "pillar_attn_unified_slotted",
            "pillar_draft_lists", "pillar_topk_workspace_bytes",
            "pillar_topk_select", "pillar_topk_select_noalloc", "pillar_get_error", "pillar_status_string",
            "pillar_kv_append", "pillar_buckets_init", "pillar_buckets_admit", "pillar_buckets_retire",
            "pillar_buckets_step", "pillar_kv_offload", "pillar_kv_reload", "pillar_offload_init",
            "pillar_attn_plan", "pillar_attn_run",
            "pillar_offload_reserve", "pillar_offload_release", "pillar_offload_evict", "pillar_offload_reload",
            "pillar_block_map_workspace_bytes", "pillar_block_map", "pillar_kv8_append",
            "pillar_attn_kv8", "pillar_attn_run_kv8",
            "pillar_prompt_attn_workspace_bytes", "pillar_prompt_attn",
            "pillar_kv8_read", "pillar_kv4_append", "pillar_kv4_read", "pillar_attn_kv4", "pillar_attn_run_kv4")
MAX_BUCKETS = 64  # PILLAR_MAX_BUCKETS
OFFLOAD_QUEUE = 1024  # PILLAR_OFFLOAD_QUEUE
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024 + 256


class PillarShape(ctypes.Structure):
    """Mirror of ``pillar_shape_t``."""
    _fields_ = [
        ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
        ("k", ctypes.c_int32), ("max_sparse", ctypes.c_int32), ("max_len", ctypes.c_int32),
        ("row_lo", ctypes.c_int32), ("row_hi", ctypes.c_int32), ("max_topk", ctypes.c_int32),
        ("verify_chunk", ctypes.c_int32), ("draft_chunk", ctypes.c_int32), ("num_slots", ctypes.c_int64),
        ("sm_scale", ctypes.c_float), ("schedule", ctypes.c_int32),
        ("wait_timeout_us", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


def make_shape(*, B, Hq, Hkv, D, k, max_sparse, max_len, num_slots, max_topk=1, row_lo=1, row_hi=None,
               verify_chunk=0, draft_chunk=0, sm_scale=0.0, schedule=0, wait_timeout_us=0) -> PillarShape:
    return PillarShape(B=B, Hq=Hq, Hkv=Hkv, D=D, k=k, max_sparse=max_sparse, max_len=max_len,
                       row_lo=row_lo, row_hi=(k + 1) if row_hi is None else row_hi, max_topk=max(1, max_topk),
                       verify_chunk=verify_chunk, draft_chunk=draft_chunk, num_slots=num_slots,
                       sm_scale=sm_scale, schedule=schedule, wait_timeout_us=wait_timeout_us)


class PillarOffloadChunk(ctypes.Structure):
    """pillar_offload_chunk_t: one chunk of an offloaded request's positions."""
    _fields_ = [("req", ctypes.c_int32), ("first", ctypes.c_int32), ("n", ctypes.c_int32), ("last", ctypes.c_int32)]


class PillarOffloadFifo(ctypes.Structure):
    """pillar_offload_fifo_t: resident slot count and the queue of offloaded chunks."""
    _fields_ = [("capacity", ctypes.c_int64), ("resident", ctypes.c_int64), ("chunk", ctypes.c_int32),
                ("head", ctypes.c_int32), ("count", ctypes.c_int32), ("pad", ctypes.c_int32),
                ("q", PillarOffloadChunk * OFFLOAD_QUEUE)]


class PillarBuckets(ctypes.Structure):
    """pillar_buckets_t: the request count of each of the k+1 phase buckets."""
    _fields_ = [("nbuckets", ctypes.c_int32), ("count", ctypes.c_int32 * MAX_BUCKETS)]


class PillarError(RuntimeError):
    def __init__(self, fn, status, flags=None):
        self.status = status
        self.flags = flags
        msg = f"{fn}: status {status} ({pillar_status_string(status)})"
        if flags is not None:
            msg += f", device flags 0x{flags:x}"
        super().__init__(msg)


_lib = None


def library_path() -> str:
    return _build.LIB


def build(force: bool = False) -> str:
    return _build.build(force=force)


def load():
    """Load the CUDA library (built in-tree by ``build()``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"the sm_103a library is not built ({path}); run __graft_entry__.build()")
    import torch  # noqa: F401  -- makes the CUDA runtime of the process available first
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    SP = ctypes.POINTER(PillarShape)
    lib.pillar_attn_workspace_bytes.argtypes = [SP, ctypes.POINTER(ctypes.c_size_t)]
    lib.pillar_attn_unified.argtypes = [SP] + [P] * 11 + [P, ctypes.c_size_t, P]
    lib.pillar_attn_unified_slotted.argtypes = [SP] + [P] * 12 + [P, ctypes.c_size_t, P]
    lib.pillar_draft_lists.argtypes = [SP, ctypes.c_int32] + [P] * 11
    lib.pillar_attn_plan.argtypes = [SP, P, P, P, P, ctypes.c_size_t, P]
    lib.pillar_attn_run.argtypes = [SP] + [P] * 10 + [ctypes.c_size_t, P]
    lib.pillar_topk_workspace_bytes.argtypes = [SP, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
    lib.pillar_topk_select.argtypes = [SP, ctypes.c_int32] + [P] * 7 + [P, ctypes.c_size_t, P]
    lib.pillar_topk_select_noalloc.argtypes = [SP, ctypes.c_int32] + [P] * 8 + [P]
    lib.pillar_get_error.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
    lib.pillar_status_string.argtypes = [ctypes.c_int]
    lib.pillar_kv_append.argtypes = [SP, P, P, P, ctypes.c_int32, P, P, P, P]
    BP = ctypes.POINTER(PillarBuckets)
    I32P = ctypes.POINTER(ctypes.c_int32)
    lib.pillar_buckets_init.argtypes = [BP, ctypes.c_int32]
    lib.pillar_buckets_admit.argtypes = [BP, I32P]
    lib.pillar_buckets_retire.argtypes = [BP, ctypes.c_int32]
    lib.pillar_buckets_step.argtypes = [BP, I32P, ctypes.c_int32, ctypes.c_int64, I32P, I32P,
                                        ctypes.POINTER(ctypes.c_int64)]
    lib.pillar_kv_offload.argtypes = [SP, P, P, P, ctypes.c_int32, P, P, P, P]
    lib.pillar_kv_reload.argtypes = [SP, P, P, P, ctypes.c_int32, P, P, P, P]
    FP = ctypes.POINTER(PillarOffloadFifo)
    lib.pillar_offload_init.argtypes = [FP, ctypes.c_int64, ctypes.c_int32]
    lib.pillar_offload_reserve.argtypes = [FP, ctypes.c_int64, ctypes.c_int32, I32P]
    lib.pillar_offload_release.argtypes = [FP, ctypes.c_int64]
    lib.pillar_offload_evict.argtypes = [FP, ctypes.c_int32, ctypes.c_int32, I32P]
    lib.pillar_offload_reload.argtypes = [FP, ctypes.POINTER(PillarOffloadChunk), ctypes.c_int32, I32P]
    I32, I64, SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.pillar_block_map_workspace_bytes.argtypes = [SP, ctypes.POINTER(SZ)]
    lib.pillar_block_map.argtypes = [SP, P, P, P, I32, P, P, P, P, P, I64, P, P, I64, P, SZ, P]
    lib.pillar_kv8_append.argtypes = [SP, P, I64, P, I64, I32, P, P, P, I32, P, P, P, P, P, P]
    lib.pillar_attn_kv8.argtypes = [SP] + [P] * 6 + [I32] + [P] * 8 + [SZ, P]
    lib.pillar_attn_run_kv8.argtypes = [SP] + [P] * 6 + [I32] + [P] * 5 + [SZ, P]
    for fmt in ("kv4", "kv8"):
        getattr(lib, f"pillar_{fmt}_read").argtypes = [SP, P, P, P, P, P, I32, P, P, I32, P, I64, P, I64, P, P]
    lib.pillar_kv4_append.argtypes = lib.pillar_kv8_append.argtypes
    lib.pillar_attn_kv4.argtypes = lib.pillar_attn_kv8.argtypes
    lib.pillar_attn_run_kv4.argtypes = lib.pillar_attn_run_kv8.argtypes
    lib.pillar_prompt_attn_workspace_bytes.argtypes = [SP, I32, ctypes.POINTER(SZ)]
    lib.pillar_prompt_attn.argtypes = [SP, P, I64, P, I64, P, I64, I32, P, P, P, P, SZ, P]
    lib.pillar_status_string.restype = ctypes.c_char_p
    for n in EXPORTED:
        if n == "pillar_status_string":
            continue
        getattr(lib, n).restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(x):
    """Device pointer of a CUDA tensor (or a raw int pointer, or None)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("device tensors only")
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return x.data_ptr()


def _nbytes(x):
    if isinstance(x, int):
        raise ValueError("a raw workspace pointer needs an explicit size")
    return x.numel() * x.element_size()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def pillar_status_string(status: int) -> str:
    if _lib is None:
        try:
            load()
        except Exception:  # pragma: no cover
            return "library not loaded"
    return _lib.pillar_status_string(int(status)).decode()


def pillar_attn_workspace_bytes(shape: PillarShape) -> int:
    out = ctypes.c_size_t(0)
    st = load().pillar_attn_workspace_bytes(ctypes.byref(shape), ctypes.byref(out))
    if st:
        raise PillarError("pillar_attn_workspace_bytes", st)
    return int(out.value)


def pillar_attn_unified(shape, q, k_pool, v_pool, slot_table, req_mode, req_len, sparse_idx, sparse_cnt, out,
                        verify_logits, verify_lse, workspace, stream=None, ws_bytes=None):
    st = load().pillar_attn_unified(
        ctypes.byref(shape), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(slot_table), _ptr(req_mode), _ptr(req_len),
        _ptr(sparse_idx), _ptr(sparse_cnt), _ptr(out), _ptr(verify_logits), _ptr(verify_lse), _ptr(workspace),
        ws_bytes if ws_bytes is not None else _nbytes(workspace), _stream(stream))
    if st:
        raise PillarError("pillar_attn_unified", st)


def pillar_attn_unified_slotted(shape, q, k_pool, v_pool, slot_table, req_mode, req_len, sparse_idx, sparse_cnt,
                                sparse_slot, out, verify_logits, verify_lse, workspace, stream=None, ws_bytes=None):
    st = load().pillar_attn_unified_slotted(
        ctypes.byref(shape), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(slot_table), _ptr(req_mode), _ptr(req_len),
        _ptr(sparse_idx), _ptr(sparse_cnt), _ptr(sparse_slot), _ptr(out), _ptr(verify_logits), _ptr(verify_lse),
        _ptr(workspace), ws_bytes if ws_bytes is not None else _nbytes(workspace), _stream(stream))
    if st:
        raise PillarError("pillar_attn_unified_slotted", st)


def pillar_attn_plan(shape, req_mode, req_len, sparse_cnt, workspace, stream=None, ws_bytes=None):
    """The device planner alone: offsets and work items of the batch, into the workspace."""
    st = load().pillar_attn_plan(ctypes.byref(shape), _ptr(req_mode), _ptr(req_len), _ptr(sparse_cnt), _ptr(workspace),
                                 ws_bytes if ws_bytes is not None else _nbytes(workspace), _stream(stream))
    if st:
        raise PillarError("pillar_attn_plan", st)


def pillar_attn_run(shape, q, k_pool, v_pool, slot_table, sparse_idx, out, verify_logits, verify_lse, workspace,
                    sparse_slot=None, stream=None, ws_bytes=None):
    """The attention kernel and the merge on the plan in the workspace (one layer of the batch the plan describes)."""
    st = load().pillar_attn_run(
        ctypes.byref(shape), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(slot_table), _ptr(sparse_idx), _ptr(sparse_slot),
        _ptr(out), _ptr(verify_logits), _ptr(verify_lse), _ptr(workspace),
        ws_bytes if ws_bytes is not None else _nbytes(workspace), _stream(stream))
    if st:
        raise PillarError("pillar_attn_run", st)


def pillar_draft_lists(shape, V, next_idx, next_cnt, group_map, verify_len, req_len, slot_table, sparse_idx,
                       sparse_cnt, sparse_slot=None, device_flags=None, stream=None):
    """The draft step's lists (and, with sparse_slot, their slots) from a verify step's Top-K."""
    st = load().pillar_draft_lists(
        ctypes.byref(shape), int(V), _ptr(next_idx), _ptr(next_cnt), _ptr(group_map), _ptr(verify_len),
        _ptr(req_len), _ptr(slot_table), _ptr(sparse_idx), _ptr(sparse_cnt), _ptr(sparse_slot), _ptr(device_flags),
        _stream(stream))
    if st:
        raise PillarError("pillar_draft_lists", st)


def pillar_topk_workspace_bytes(shape: PillarShape, V: int) -> int:
    out = ctypes.c_size_t(0)
    st = load().pillar_topk_workspace_bytes(ctypes.byref(shape), int(V), ctypes.byref(out))
    if st:
        raise PillarError("pillar_topk_workspace_bytes", st)
    return int(out.value)


def pillar_topk_select(shape, V, verify_logits, verify_lse, req_len, group_map, K, next_idx, next_cnt, workspace,
                       stream=None, ws_bytes=None):
    st = load().pillar_topk_select(
        ctypes.byref(shape), int(V), _ptr(verify_logits), _ptr(verify_lse), _ptr(req_len), _ptr(group_map), _ptr(K),
        _ptr(next_idx), _ptr(next_cnt), _ptr(workspace), ws_bytes if ws_bytes is not None else _nbytes(workspace),
        _stream(stream))
    if st:
        raise PillarError("pillar_topk_select", st)


def pillar_topk_select_noalloc(shape, V, verify_logits, verify_lse, req_len, group_map, K, next_idx, next_cnt,
                               device_flags=None, stream=None):
    """pillar_topk_select for callers that cannot allocate device memory: the
    library's built-in scratch array replaces the workspace.  Calls sharing a
    device must not overlap on the GPU; the first call on a device should come
    before any stream capture."""
    st = load().pillar_topk_select_noalloc(
        ctypes.byref(shape), int(V), _ptr(verify_logits), _ptr(verify_lse), _ptr(req_len), _ptr(group_map), _ptr(K),
        _ptr(next_idx), _ptr(next_cnt), _ptr(device_flags), _stream(stream))
    if st:
        raise PillarError("pillar_topk_select_noalloc", st)


def pillar_get_error(workspace, stream=None) -> int:
    """Synchronise, read and clear the device error word; returns the flags."""
    flags = ctypes.c_int32(0)
    st = load().pillar_get_error(_ptr(workspace), _stream(stream), ctypes.byref(flags))
    if st not in (0, -4):
        raise PillarError("pillar_get_error", st)
    return int(flags.value)


def pillar_kv_append(shape, k_new, v_new, slots, k_pool, v_pool, device_flags=None, stream=None):
    """Scatter n new tokens' K/V rows ([n, Hkv, D] bf16) into the pools at
    slots[0..n); out-of-range slots are skipped and flagged in device_flags."""
    n = int(slots.numel()) if not isinstance(slots, int) else None
    if n is None:
        raise ValueError("slots must be a tensor (its length is the token count)")
    st = load().pillar_kv_append(ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _ptr(slots), n, _ptr(k_pool),
                                 _ptr(v_pool), _ptr(device_flags), _stream(stream))
    if st:
        raise PillarError("pillar_kv_append", st)


def _host_ptr(x):
    """Address of a host buffer for the offload copies (a CPU tensor, page-locked
    or not: the library refuses memory the device cannot address), a CUDA
    tensor, or a raw int pointer."""
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


def pillar_kv_offload(shape, k_pool, v_pool, slots, host_k, host_v, device_flags=None, stream=None):
    """Pack the slot blocks k_pool[slots[i]], v_pool[slots[i]] into rows i of
    host_k, host_v ([n, Hkv, D] bf16, page-locked host memory, e.g. a tensor
    made with pin_memory=True); out-of-range slots are skipped and flagged."""
    n = int(slots.numel())
    st = load().pillar_kv_offload(ctypes.byref(shape), _ptr(k_pool), _ptr(v_pool), _ptr(slots), n,
                                  _host_ptr(host_k), _host_ptr(host_v), _ptr(device_flags), _stream(stream))
    if st:
        raise PillarError("pillar_kv_offload", st)


def pillar_kv_reload(shape, host_k, host_v, slots, k_pool, v_pool, device_flags=None, stream=None):
    """The way back: rows i of host_k, host_v go to the slot blocks slots[i]."""
    n = int(slots.numel())
    st = load().pillar_kv_reload(ctypes.byref(shape), _host_ptr(host_k), _host_ptr(host_v), _ptr(slots), n,
                                 _ptr(k_pool), _ptr(v_pool), _ptr(device_flags), _stream(stream))
    if st:
        raise PillarError("pillar_kv_reload", st)


# --------------------------------------------------------------- cache blocks

class _Types:
    """Element types the calls below take, and torch's accessors of the current device and stream (torch is imported on
    the first use; the raw accessors cost a tenth of the objects')."""

    def __getattr__(self, name):
        import torch
        self.i32, self.i64, self.f32 = (torch.int32,), (torch.int64,), (torch.float32,)
        self.bf16 = (torch.bfloat16, torch.int16, torch.uint16)  # bf16 bits travel in 16-bit integers too
        self.codes = (torch.uint8, torch.int8, torch.float8_e4m3fn)
        self.bytes = (torch.uint8, torch.int8)
        torch.cuda.init()
        self.device, self.stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        return self.__dict__[name]


_T = _Types()


def _raw_stream(stream, dev):
    if stream is None:
        return _T.stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _misfit(name, x, dtypes, shape, dev):
    if x.dtype not in dtypes:
        raise ValueError(f"{name}: {x.dtype}, expected {' or '.join(map(str, dtypes))}")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if not x.is_cuda or x.get_device() != dev:
        raise ValueError(f"{name}: on {x.device}, expected the current CUDA device ({dev})")
    raise ValueError(f"{name}: must be contiguous")


def _arg(name, x, dtypes, shape, dev):
    """Pointer of a CUDA tensor whose element type, shape, layout and device are as given: these calls index their arrays by
    the sizes of other ones, so a tensor that does not fit is refused here."""
    if x.dtype in dtypes and x.shape == shape and x.get_device() == dev and x.is_contiguous():
        return x.data_ptr()
    _misfit(name, x, dtypes, shape, dev)


def _dim(name, x, i, ndim):
    """Extent i of a tensor whose extents the call goes by."""
    if x.ndim != ndim:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {ndim} dimensions")
    return x.shape[i]


def _dim32(name, x, i, ndim):
    """The same for an extent that the call takes as a 32-bit count (ctypes would wrap a larger one)."""
    return _count32(name, _dim(name, x, i, ndim))


def _count32(name, n):
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name}: {n}, more than a 32-bit count")
    return n


def _rows(name, x, rows, heads, D, dev):
    """Pointer and token stride of [rows, heads, D] bf16 whose tokens may lie apart (a slice of a fused projection)."""
    if x.dtype not in _T.bf16 or x.shape != (rows, heads, D) or x.get_device() != dev:
        _misfit(name, x, _T.bf16, (rows, heads, D), dev)
    if x.is_contiguous():
        return x.data_ptr(), 0
    st = x.stride()
    if st[2] != 1 or (heads > 1 and st[1] != D) or (rows > 1 and st[0] < heads * D):
        raise ValueError(f"{name}: strides {st}, expected each token's {heads} x {D} values to be contiguous")
    return x.data_ptr(), st[0] if rows > 1 else 0


def _workspace(x, dev):
    if x.get_device() != dev or not x.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the current CUDA device")
    return x.data_ptr(), x.nbytes


def pillar_block_map_workspace_bytes(shape: PillarShape) -> int:
    out = ctypes.c_size_t(0)
    st = load().pillar_block_map_workspace_bytes(ctypes.byref(shape), ctypes.byref(out))
    if st:
        raise PillarError("pillar_block_map_workspace_bytes", st)
    return int(out.value)


def pillar_block_map(shape, req_len, prev_len, block_table, free_ring, free_state, granted_len, kv_off, slot_table,
                     new_off, new_slots, workspace, stream=None):
    """Blocks for a batch whose lengths go from prev_len to req_len: takes them from and gives them back to the free
    ring, and writes the block table's new entries, the slot table and the new tokens' slots."""
    dev, B = _T.device(), shape.B
    ws, ws_bytes = _workspace(workspace, dev)
    width, slots, new = (_dim32("block_table", block_table, 1, 2), _dim("slot_table", slot_table, 0, 1),
                         _dim("new_slots", new_slots, 0, 1))
    st = load().pillar_block_map(
        ctypes.byref(shape), _arg("req_len", req_len, _T.i32, (B,), dev), _arg("prev_len", prev_len, _T.i32, (B,), dev),
        _arg("block_table", block_table, _T.i32, (B, width), dev), width,
        _arg("free_ring", free_ring, _T.i32, (shape.num_slots // KV_BLOCK,), dev),
        _arg("free_state", free_state, _T.i32, (2,), dev), _arg("granted_len", granted_len, _T.i32, (B,), dev),
        _arg("kv_off", kv_off, _T.i64, (B + 1,), dev), _arg("slot_table", slot_table, _T.i32, (slots,), dev), slots,
        _arg("new_off", new_off, _T.i32, (B + 1,), dev),
        _arg("new_slots", new_slots, _T.i32, (new,), dev), new, ws, ws_bytes, _raw_stream(stream, dev))
    if st:
        raise PillarError("pillar_block_map", st)


def _pool8(shape, k8_pool, v8_pool, k_scale, v_scale, dev):
    blocks = (shape.num_slots // KV_BLOCK, shape.Hkv)
    return (_arg("k8_pool", k8_pool, _T.codes, blocks + (KV_BLOCK, shape.D), dev),
            _arg("v8_pool", v8_pool, _T.codes, blocks + (KV_BLOCK, shape.D), dev),
            _arg("k_scale", k_scale, _T.f32, blocks, dev), _arg("v_scale", v_scale, _T.f32, blocks, dev))


def _pool4(shape, k4_pool, v4_pool, k_scale, v_scale, dev):
    rows = (shape.num_slots // KV_BLOCK, shape.Hkv, KV_BLOCK)
    codes, groups = rows + (shape.D // 2,), rows + (shape.D // KV4_GROUP,)
    return (_arg("k4_pool", k4_pool, _T.bytes, codes, dev), _arg("v4_pool", v4_pool, _T.bytes, codes, dev),
            _arg("k_scale", k_scale, _T.bytes, groups, dev), _arg("v_scale", v_scale, _T.bytes, groups, dev))


def pillar_kv8_append(shape, k_new, v_new, req_len, new_off, block_table, k8_pool, v8_pool, k_scale, v_scale,
                      device_flags=None, stream=None):
    """The new tokens' K/V rows ([n, Hkv, D] bf16, tokens may lie apart) as e4m3 codes under the scales of their blocks;
    request b's rows new_off[b] .. new_off[b+1]-1 are its last positions."""
    _append("pillar_kv8_append", _pool8, shape, k_new, v_new, req_len, new_off, block_table,
            (k8_pool, v8_pool, k_scale, v_scale), device_flags, stream)


def pillar_kv4_append(shape, k_new, v_new, req_len, new_off, block_table, k4_pool, v4_pool, k_scale, v_scale,
                      device_flags=None, stream=None):
    """The same into the 4-bit cache: e2m1 codes and a scale byte for every 16 values of a row."""
    _append("pillar_kv4_append", _pool4, shape, k_new, v_new, req_len, new_off, block_table,
            (k4_pool, v4_pool, k_scale, v_scale), device_flags, stream)


def _append(name, pool, shape, k_new, v_new, req_len, new_off, block_table, cache, device_flags, stream):
    dev, B = _T.device(), shape.B
    n, width = _dim32("k_new", k_new, 0, 3), _dim32("block_table", block_table, 1, 2)
    kp, ks = _rows("k_new", k_new, n, shape.Hkv, shape.D, dev)
    vp, vs = _rows("v_new", v_new, n, shape.Hkv, shape.D, dev)
    st = getattr(load(), name)(
        ctypes.byref(shape), kp, ks, vp, vs, n, _arg("req_len", req_len, _T.i32, (B,), dev),
        _arg("new_off", new_off, _T.i32, (B + 1,), dev), _arg("block_table", block_table, _T.i32, (B, width), dev),
        width, *pool(shape, *cache, dev),
        None if device_flags is None else _arg("device_flags", device_flags, _T.i32, (1,), dev),
        _raw_stream(stream, dev))
    if st:
        raise PillarError(name, st)


def pillar_kv8_read(shape, k8_pool, v8_pool, k_scale, v_scale, block_table, first, out_off, k_out, v_out,
                    device_flags=None, stream=None):
    """Positions of the 8-bit cache as bf16 rows ([n, Hkv, D], tokens may lie apart): rows out_off[b] .. out_off[b+1]-1 are
    the positions of request b from first[b] on."""
    _read("pillar_kv8_read", _pool8, shape, (k8_pool, v8_pool, k_scale, v_scale), block_table, first, out_off, k_out, v_out,
          device_flags, stream)


def pillar_kv4_read(shape, k4_pool, v4_pool, k_scale, v_scale, block_table, first, out_off, k_out, v_out,
                    device_flags=None, stream=None):
    """The same out of the 4-bit cache."""
    _read("pillar_kv4_read", _pool4, shape, (k4_pool, v4_pool, k_scale, v_scale), block_table, first, out_off, k_out, v_out,
          device_flags, stream)


def _read(name, pool, shape, cache, block_table, first, out_off, k_out, v_out, device_flags, stream):
    dev, B = _T.device(), shape.B
    n, width = _dim32("k_out", k_out, 0, 3), _dim32("block_table", block_table, 1, 2)
    kp, ks = _rows("k_out", k_out, n, shape.Hkv, shape.D, dev)
    vp, vs = _rows("v_out", v_out, n, shape.Hkv, shape.D, dev)
    st = getattr(load(), name)(
        ctypes.byref(shape), *pool(shape, *cache, dev), _arg("block_table", block_table, _T.i32, (B, width), dev), width,
        _arg("first", first, _T.i32, (B,), dev), _arg("out_off", out_off, _T.i32, (B + 1,), dev), n, kp, ks, vp, vs,
        None if device_flags is None else _arg("device_flags", device_flags, _T.i32, (1,), dev),
        _raw_stream(stream, dev))
    if st:
        raise PillarError(name, st)


def _attn_cache_args(shape, q, pool, cache, block_table, dev):
    width = _dim32("block_table", block_table, 1, 2)
    return (_arg("q", q, _T.bf16, (_dim("q", q, 0, 3), shape.Hq, shape.D), dev), *pool(shape, *cache, dev),
            _arg("block_table", block_table, _T.i32, (shape.B, width), dev), width)


def _attn_cache_outputs(shape, q, out, verify_logits, verify_lse, workspace, dev):
    return (_arg("out", out, _T.bf16, q.shape, dev),
            None if verify_logits is None else
            _arg("verify_logits", verify_logits, _T.f32, (_dim("verify_logits", verify_logits, 0, 1),), dev),
            _arg("verify_lse", verify_lse, _T.f32, (_dim("verify_lse", verify_lse, 0, 3), shape.Hq, shape.k + 1), dev),
            *_workspace(workspace, dev))


def _attn_cache(name, pool, shape, q, cache, block_table, req_mode, req_len, sparse_idx, sparse_cnt, out, verify_logits,
                verify_lse, workspace, stream):
    dev, B = _T.device(), shape.B
    st = getattr(load(), name)(
        ctypes.byref(shape), *_attn_cache_args(shape, q, pool, cache, block_table, dev),
        _arg("req_mode", req_mode, _T.i32, (B,), dev), _arg("req_len", req_len, _T.i32, (B,), dev),
        _arg("sparse_idx", sparse_idx, _T.i32, (B, shape.Hkv, shape.max_sparse), dev),
        _arg("sparse_cnt", sparse_cnt, _T.i32, (B, shape.Hkv), dev),
        *_attn_cache_outputs(shape, q, out, verify_logits, verify_lse, workspace, dev), _raw_stream(stream, dev))
    if st:
        raise PillarError(name, st)


def _attn_run_cache(name, pool, shape, q, cache, block_table, sparse_idx, out, verify_logits, verify_lse, workspace, stream):
    dev = _T.device()
    st = getattr(load(), name)(
        ctypes.byref(shape), *_attn_cache_args(shape, q, pool, cache, block_table, dev),
        _arg("sparse_idx", sparse_idx, _T.i32, (shape.B, shape.Hkv, shape.max_sparse), dev),
        *_attn_cache_outputs(shape, q, out, verify_logits, verify_lse, workspace, dev), _raw_stream(stream, dev))
    if st:
        raise PillarError(name, st)


def pillar_attn_kv8(shape, q, k8_pool, v8_pool, k_scale, v_scale, block_table, req_mode, req_len, sparse_idx, sparse_cnt,
                    out, verify_logits, verify_lse, workspace, stream=None):
    """The unified draft/verify step over the 8-bit cache; verify_logits None: no dump.  (The sizes of q, out, the logits
    and the LSEs follow from modes and lengths that only the device knows, as in pillar_attn_unified.)"""
    _attn_cache("pillar_attn_kv8", _pool8, shape, q, (k8_pool, v8_pool, k_scale, v_scale), block_table, req_mode, req_len,
                sparse_idx, sparse_cnt, out, verify_logits, verify_lse, workspace, stream)


def pillar_attn_run_kv8(shape, q, k8_pool, v8_pool, k_scale, v_scale, block_table, sparse_idx, out, verify_logits,
                        verify_lse, workspace, stream=None):
    """pillar_attn_kv8 on the plan that pillar_attn_plan left in the workspace."""
    _attn_run_cache("pillar_attn_run_kv8", _pool8, shape, q, (k8_pool, v8_pool, k_scale, v_scale), block_table, sparse_idx,
                    out, verify_logits, verify_lse, workspace, stream)


def pillar_attn_kv4(shape, q, k4_pool, v4_pool, k_scale, v_scale, block_table, req_mode, req_len, sparse_idx, sparse_cnt,
                    out, verify_logits, verify_lse, workspace, stream=None):
    """The unified draft/verify step over the 4-bit cache; verify_logits None: no dump."""
    _attn_cache("pillar_attn_kv4", _pool4, shape, q, (k4_pool, v4_pool, k_scale, v_scale), block_table, req_mode, req_len,
                sparse_idx, sparse_cnt, out, verify_logits, verify_lse, workspace, stream)


def pillar_attn_run_kv4(shape, q, k4_pool, v4_pool, k_scale, v_scale, block_table, sparse_idx, out, verify_logits,
                        verify_lse, workspace, stream=None):
    """pillar_attn_kv4 on the plan that pillar_attn_plan left in the workspace."""
    _attn_run_cache("pillar_attn_run_kv4", _pool4, shape, q, (k4_pool, v4_pool, k_scale, v_scale), block_table, sparse_idx,
                    out, verify_logits, verify_lse, workspace, stream)


# --------------------------------------------------------------- prompts

def pillar_prompt_attn_workspace_bytes(shape: PillarShape, n: int) -> int:
    out = ctypes.c_size_t(0)
    st = load().pillar_prompt_attn_workspace_bytes(ctypes.byref(shape), _count32("n", int(n)), ctypes.byref(out))
    if st:
        raise PillarError("pillar_prompt_attn_workspace_bytes", st)
    return int(out.value)


def pillar_prompt_attn(shape, q, k, v, seq_off, out, lse, workspace, stream=None):
    """Causal attention over prompts packed one after another ([n, heads, D] bf16; tokens may lie apart); lse [n, Hq] fp32
    or None."""
    dev, n = _T.device(), _dim32("q", q, 0, 3)
    qp, qs = _rows("q", q, n, shape.Hq, shape.D, dev)
    kp, ks = _rows("k", k, n, shape.Hkv, shape.D, dev)
    vp, vs = _rows("v", v, n, shape.Hkv, shape.D, dev)
    st = load().pillar_prompt_attn(
        ctypes.byref(shape), qp, qs, kp, ks, vp, vs, n, _arg("seq_off", seq_off, _T.i32, (shape.B + 1,), dev),
        _arg("out", out, _T.bf16, (n, shape.Hq, shape.D), dev),
        None if lse is None else _arg("lse", lse, _T.f32, (n, shape.Hq), dev), *_workspace(workspace, dev),
        _raw_stream(stream, dev))
    if st:
        raise PillarError("pillar_prompt_attn", st)


# --------------------------------------------------------------- offload FIFO (host side)

def pillar_offload_init(capacity: int, chunk: int) -> PillarOffloadFifo:
    f = PillarOffloadFifo()
    st = load().pillar_offload_init(ctypes.byref(f), int(capacity), int(chunk))
    if st:
        raise PillarError("pillar_offload_init", st)
    return f


def pillar_offload_reserve(f: PillarOffloadFifo, n: int, new_request: bool) -> bool:
    """True if n more device slots were granted (see the header)."""
    g = ctypes.c_int32(0)
    st = load().pillar_offload_reserve(ctypes.byref(f), int(n), 1 if new_request else 0, ctypes.byref(g))
    if st:
        raise PillarError("pillar_offload_reserve", st)
    return bool(g.value)


def pillar_offload_release(f: PillarOffloadFifo, n: int) -> None:
    st = load().pillar_offload_release(ctypes.byref(f), int(n))
    if st:
        raise PillarError("pillar_offload_release", st)


def pillar_offload_evict(f: PillarOffloadFifo, req: int, length: int) -> int:
    """Queue request `req`'s positions [0, length) for the host; returns its chunk count."""
    nc = ctypes.c_int32(0)
    st = load().pillar_offload_evict(ctypes.byref(f), int(req), int(length), ctypes.byref(nc))
    if st:
        raise PillarError("pillar_offload_evict", st)
    return int(nc.value)


def pillar_offload_reload(f: PillarOffloadFifo, max_out: int = OFFLOAD_QUEUE):
    """Chunks to bring back now, as (req, first, n, last) tuples, oldest requests first."""
    out = (PillarOffloadChunk * max(1, max_out))()
    nout = ctypes.c_int32(0)
    st = load().pillar_offload_reload(ctypes.byref(f), out, int(max_out), ctypes.byref(nout))
    if st:
        raise PillarError("pillar_offload_reload", st)
    return [(c.req, c.first, c.n, c.last) for c in out[:nout.value]]


# --------------------------------------------------------------- phase buckets (host side)

def pillar_buckets_init(k: int) -> PillarBuckets:
    pb = PillarBuckets()
    st = load().pillar_buckets_init(ctypes.byref(pb), int(k))
    if st:
        raise PillarError("pillar_buckets_init", st)
    return pb


def pillar_buckets_admit(pb: PillarBuckets) -> int:
    """Bucket of a new request (the least loaded one, lowest index among equals)."""
    b = ctypes.c_int32(-1)
    st = load().pillar_buckets_admit(ctypes.byref(pb), ctypes.byref(b))
    if st:
        raise PillarError("pillar_buckets_admit", st)
    return int(b.value)


def pillar_buckets_retire(pb: PillarBuckets, bucket: int) -> None:
    st = load().pillar_buckets_retire(ctypes.byref(pb), int(bucket))
    if st:
        raise PillarError("pillar_buckets_retire", st)


def pillar_buckets_step(pb: PillarBuckets, buckets, step: int):
    """(req_mode, phase, q_rows) of the requests with these buckets at `step`
    (lists of ints and the step's query-row count)."""
    n = len(buckets)
    arr = (ctypes.c_int32 * max(1, n))(*buckets)
    mode = (ctypes.c_int32 * max(1, n))()
    phase = (ctypes.c_int32 * max(1, n))()
    rows = ctypes.c_int64(0)
    st = load().pillar_buckets_step(ctypes.byref(pb), arr, n, int(step), mode, phase, ctypes.byref(rows))
    if st:
        raise PillarError("pillar_buckets_step", st)
    return list(mode)[:n], list(phase)[:n], int(rows.value)
