"""Python binding of libdsa, the GB300 DeepSeek-Sparse-Attention hot path.

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libdsa.so`` behind the C ABI declared in ``include/dsa.h``.  The functions
below keep the C names, take torch CUDA tensors (PyTorch supplies device
memory and streams), pass their raw device pointers through ``ctypes`` and
raise :class:`DsaError` on any non-OK status.  There is no fallback: if the
library is missing or fails to load, importing the entry points raises.

Tensor layouts (row-major, contiguous), with ``W = kv_lora + rope_dim``:

* ``q_idx`` [n_q, idx_heads, idx_dim], ``k_idx`` [keys, idx_dim],
  ``q_abs`` [n_q, heads, W], ``cache`` [rows, W]: float32 or bfloat16
  (one dtype for all four, the shape's ``dtype``)
* ``w`` [n_q, idx_heads] float32
* ``scores`` [n_q, ld] float32, ``idx`` [n_q, top_k + kpool - 1] int32,
  ``n_sel`` [n_q] int32, ``out`` [n_q, heads, kv_lora] float32,
  ``lse`` [n_q, heads] float32
* ``q`` [n_q, heads, nope + rope], ``k_nope`` [rows, heads, nope], ``v`` and ``out`` of the
  expanded attention [.., heads, v_dim]: the shape's dtype
* ``dsa_rms_norm`` and ``dsa_rope`` also take tensors whose rows (and heads) are parts of
  wider ones; their last dimension has stride 1
* the paged 8-bit cache: ``codes`` [n_pages, page_rows, W] of one-byte elements,
  ``scales`` [n_pages, 2] uint8 ([n_pages, 1] without rope), ``block_table``
  [n_seq, table_ld] int32, ``slots`` [tokens] int64
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

__all__ = [
    "DsaError", "Shape", "Batch", "load", "make_shape", "make_batch", "workspace_size",
    "alloc_workspace", "dsa_version", "dsa_index_row_width", "dsa_workspace_size",
    "dsa_workspace_init", "dsa_plan", "dsa_index_scores", "dsa_topk_select", "dsa_index_select",
    "dsa_sparse_mla_attn",
    "dsa_decode_step", "dsa_decode_step_host", "dsa_decode_step_noalloc", "dsa_check_device_error", "DecodeStep", "LIB_PATH",
    "OP_INDEX_SCORES", "OP_TOPK_SELECT", "OP_SPARSE_MLA", "OP_DECODE_STEP", "OP_INDEX_SELECT",
    "OP_POOL_COMPRESS", "dsa_pool_compress", "dsa_index_prepare", "dsa_workspace_set_wait_budget",
    "FLAG_TWO_LAUNCH", "FLAG_DESC_ORDER", "FLAG_DENSE", "OP_PROJECT", "dsa_absorb_q",
    "dsa_up_project", "OP_DECODE_STEP_HOST",
    "Pages", "make_pages", "CACHE_E4M3", "CACHE_S8", "OP_PAGE_PLAN", "OP_CACHE_APPEND",
    "OP_PAGED_MLA", "dsa_page_plan", "dsa_cache_append", "dsa_paged_mla_attn",
    "RopePlan", "make_rope", "ROPE_PAIRS", "ROPE_HALVES", "NORM_SAME", "NORM_E4M3",
    "OP_EXPANDED_MLA", "dsa_rms_norm", "dsa_rope_init", "dsa_rope", "dsa_expand_kv",
    "dsa_expanded_mla_attn",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdsa.so")

DSA_F32, DSA_BF16 = 0, 1
OP_INDEX_SCORES, OP_TOPK_SELECT, OP_SPARSE_MLA, OP_DECODE_STEP, OP_INDEX_SELECT = 0, 1, 2, 3, 4
OP_POOL_COMPRESS = 5
OP_PROJECT = 6
OP_DECODE_STEP_HOST = 7
OP_PAGE_PLAN, OP_CACHE_APPEND, OP_PAGED_MLA = 16, 17, 18
OP_EXPANDED_MLA = 24
CACHE_E4M3, CACHE_S8 = 0, 1
NORM_SAME, NORM_E4M3 = 0, 1
ROPE_PAIRS, ROPE_HALVES, ROPE_MAX_PAIRS = 0, 1, 128
FLAG_TWO_LAUNCH, FLAG_DESC_ORDER, FLAG_DENSE = 0x1, 0x2, 0x4
_TORCH_DTYPE = {DSA_F32: torch.float32, DSA_BF16: torch.bfloat16}
STATUS = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED",
          3: "DSA_ERR_WORKSPACE", 4: "DSA_ERR_CUDA", 5: "DSA_ERR_DEVICE", 6: "DSA_ERR_TIMEOUT"}


class DsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")


class Shape(ctypes.Structure):
    _fields_ = [("idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("kv_lora", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("kpool", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class Batch(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_q", ctypes.c_int32),
                ("max_q_len", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("max_kv_len", ctypes.c_int64), ("total_rows", ctypes.c_int64),
                ("total_keys", ctypes.c_int64), ("row_off", ctypes.c_void_p),
                ("key_off", ctypes.c_void_p), ("q_off", ctypes.c_void_p)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("kernel_launches", ctypes.c_int32), ("attn_splits", ctypes.c_int32),
                ("attn_rows_per_split", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Pages(ctypes.Structure):
    _fields_ = [("page_rows", ctypes.c_int32), ("format", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("table_ld", ctypes.c_int64)]


class RopePlan(ctypes.Structure):
    _fields_ = [("dims", ctypes.c_int32), ("layout", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("turns", ctypes.c_uint64 * ROPE_MAX_PAIRS)]


_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Load libdsa.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdsa.so not found at {LIB_PATH}: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        P, S, i32, i64, sz = (ctypes.c_void_p, ctypes.POINTER(Shape), ctypes.c_int32,
                              ctypes.c_int64, ctypes.c_size_t)
        B = ctypes.POINTER(Batch)
        G = ctypes.POINTER(Pages)
        R = ctypes.POINTER(RopePlan)
        sigs = {
            "dsa_version": ([], ctypes.c_int),
            "dsa_status_string": ([i32], ctypes.c_char_p),
            "dsa_index_row_width": ([S], i64),
            "dsa_workspace_size": ([S, B, i32, ctypes.POINTER(sz)], ctypes.c_int),
            "dsa_workspace_init": ([P, sz, P], ctypes.c_int),
            "dsa_plan": ([S, B, i32, ctypes.POINTER(PlanInfo)], ctypes.c_int),
            "dsa_index_scores": ([S, B, P, P, P, P, i64, P, sz, P], ctypes.c_int),
            "dsa_topk_select": ([S, B, P, i64, P, P, P, sz, P], ctypes.c_int),
            "dsa_index_select": ([S, B, P, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_sparse_mla_attn": ([S, B, P, P, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_decode_step": ([S, B, P, P, P, P, P, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_decode_step_host": ([S, B, P, P, P, P, P, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_check_device_error": ([P, sz, P, ctypes.POINTER(i32)], ctypes.c_int),
            "dsa_decode_step_noalloc": ([S, B, P, P, P, P, P, P, P, P, P, P], ctypes.c_int),
            "dsa_pool_compress": ([S, B, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_index_prepare": ([S, i64, P, P, i32, ctypes.c_double, P, P], ctypes.c_int),
            "dsa_workspace_set_wait_budget": ([P, sz, ctypes.c_uint64, P], ctypes.c_int),
            "dsa_absorb_q": ([S, i32, i32, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_up_project": ([S, i32, i32, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_page_plan": ([G, i32, i64, P, P, P, P, P, P, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_cache_append": ([S, B, G, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_rms_norm": ([i64, i32, i32, P, i64, P, i64, P, ctypes.c_float, P, i64, P, i64, i32, P,
                              i32, P], ctypes.c_int),
            "dsa_rope_init": ([R, i32, i32, i32] + [ctypes.c_double] * 6, ctypes.c_int),
            "dsa_rope": ([R, i32, i64, i32, P, i64, i64, P, P, i64, i64, P], ctypes.c_int),
            "dsa_expand_kv": ([S, i64, i32, i32, P, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_expanded_mla_attn": ([S, B, i32, i32, P, P, P, P, P, P, P, sz, P], ctypes.c_int),
            "dsa_paged_mla_attn": ([S, B, G, P, P, P, P, P, P, P, P, P, sz, P], ctypes.c_int),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libdsa takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libdsa takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle; torch.cuda.current_stream() wraps it in an object,
# which costs a microsecond or more per call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _call(name: str, *args) -> int:
    rc = getattr(_lib or load(), name)(*args)
    if rc != 0:
        raise DsaError(name, rc)
    return rc


def make_shape(idx_heads=32, idx_dim=128, heads=64, kv_lora=512, rope_dim=64, top_k=2048,
               kpool=1, scale=1.0 / 16.0, dtype="bf16") -> Shape:
    d = {"f32": DSA_F32, "bf16": DSA_BF16, torch.float32: DSA_F32, torch.bfloat16: DSA_BF16}[dtype]
    return Shape(idx_heads, idx_dim, heads, kv_lora, rope_dim, top_k, kpool, float(scale), d)


def make_batch(row_off: torch.Tensor, key_off: torch.Tensor, q_off: torch.Tensor, n_q: int,
               max_q_len: int, max_kv_len: int, total_rows: int, total_keys: int,
               flags: int = 0) -> Batch:
    """Batch descriptor over int64 device offset arrays of n_seq+1 entries.

    ``total_rows`` / ``total_keys`` are the row counts of the cache and key
    tensors; ``flags`` the call's ``FLAG_*`` options.  The returned structure
    holds raw pointers: keep the three tensors alive while it is in use.
    """
    for t in (row_off, key_off, q_off):
        if t.dtype != torch.int64:
            raise ValueError("offset arrays are int64")
    n_seq = row_off.numel() - 1
    b = Batch(n_seq, int(n_q), int(max_q_len), int(flags), int(max_kv_len), int(total_rows),
              int(total_keys), _ptr(row_off), _ptr(key_off), _ptr(q_off))
    b._keep = (row_off, key_off, q_off)
    return b


def dsa_version() -> int:
    return load().dsa_version()


def dsa_index_row_width(shape: Shape) -> int:
    return int(load().dsa_index_row_width(ctypes.byref(shape)))


def dsa_workspace_size(shape: Shape, batch: Batch, op: int) -> int:
    n = ctypes.c_size_t(0)
    _call("dsa_workspace_size", ctypes.byref(shape), ctypes.byref(batch), op, ctypes.byref(n))
    return int(n.value)


workspace_size = dsa_workspace_size


def dsa_plan(shape: Shape, batch: Batch, op: int) -> dict:
    info = PlanInfo()
    _call("dsa_plan", ctypes.byref(shape), ctypes.byref(batch), op, ctypes.byref(info))
    return {"kernel_launches": info.kernel_launches, "attn_splits": info.attn_splits,
            "attn_rows_per_split": info.attn_rows_per_split}


def alloc_workspace(shape: Shape, batch: Batch, op: int = OP_DECODE_STEP,
                    device="cuda") -> torch.Tensor:
    """Zero-filled workspace of the size the library asks for (256-byte aligned)."""
    n = dsa_workspace_size(shape, batch, op)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def dsa_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _call("dsa_workspace_init", _ptr(ws), ws.numel(), _stream(stream))


def dsa_index_scores(shape, batch, q_idx, w, k_idx, scores, ld, ws, stream=None) -> None:
    _call("dsa_index_scores", ctypes.byref(shape), ctypes.byref(batch), _ptr(q_idx), _ptr(w),
          _ptr(k_idx), _ptr(scores), int(ld), _ptr(ws), ws.numel(), _stream(stream))


def dsa_topk_select(shape, batch, scores, ld, idx, n_sel, ws, stream=None) -> None:
    _call("dsa_topk_select", ctypes.byref(shape), ctypes.byref(batch), _ptr(scores), int(ld),
          _ptr(idx), _ptr(n_sel), _ptr(ws), ws.numel(), _stream(stream))


def dsa_index_select(shape, batch, q_idx, w, k_idx, idx, n_sel, ws, stream=None) -> None:
    _call("dsa_index_select", ctypes.byref(shape), ctypes.byref(batch), _ptr(q_idx), _ptr(w),
          _ptr(k_idx), _ptr(idx), _ptr(n_sel), _ptr(ws), ws.numel(), _stream(stream))


def dsa_sparse_mla_attn(shape, batch, q_abs, cache, idx, n_sel, out, lse, ws, stream=None) -> None:
    _call("dsa_sparse_mla_attn", ctypes.byref(shape), ctypes.byref(batch), _ptr(q_abs),
          _ptr(cache), _ptr(idx), _ptr(n_sel), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
          _stream(stream))


def dsa_decode_step(shape, batch, q_idx, w, k_idx, q_abs, cache, out, lse=None, idx_out=None,
                    n_sel_out=None, ws=None, stream=None) -> None:
    _call("dsa_decode_step", ctypes.byref(shape), ctypes.byref(batch), _ptr(q_idx), _ptr(w),
          _ptr(k_idx), _ptr(q_abs), _ptr(cache), _ptr(out), _ptr(lse), _ptr(idx_out),
          _ptr(n_sel_out), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream))


def _host_ptr(t: Optional[torch.Tensor]):
    """A pinned host tensor's address (or a CUDA tensor's): the per-step
    buffers of dsa_decode_step_host."""
    if t is None:
        return None
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError("dsa_decode_step_host takes pinned host (or CUDA) tensors")
    if not t.is_contiguous():
        raise ValueError("libdsa takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def dsa_decode_step_host(shape, batch, q_idx, w, k_idx, q_abs, cache, out, lse=None,
                         idx_out=None, n_sel_out=None, ws=None, stream=None) -> None:
    """dsa_decode_step with q_idx, w, q_abs, out and lse in page-locked host
    memory (or device memory); the workspace is sized with OP_DECODE_STEP_HOST."""
    _call("dsa_decode_step_host", ctypes.byref(shape), ctypes.byref(batch), _host_ptr(q_idx),
          _host_ptr(w), _ptr(k_idx), _host_ptr(q_abs), _ptr(cache), _host_ptr(out),
          _host_ptr(lse), _ptr(idx_out),
          _ptr(n_sel_out), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream))


def dsa_decode_step_noalloc(shape, batch, q_idx, w, k_idx, q_abs, cache, out, lse=None,
                            idx_out=None, n_sel_out=None, stream=None) -> None:
    """dsa_decode_step without a workspace, for callers that cannot allocate
    device memory: the scratch is a fixed array inside libdsa (see dsa.h)."""
    _call("dsa_decode_step_noalloc", ctypes.byref(shape), ctypes.byref(batch), _ptr(q_idx),
          _ptr(w), _ptr(k_idx), _ptr(q_abs), _ptr(cache), _ptr(out), _ptr(lse), _ptr(idx_out),
          _ptr(n_sel_out), _stream(stream))


def dsa_pool_compress(shape, batch, cells, pos, pool_keys, ws, stream=None) -> None:
    """Compressed keys of the pools completed by each sequence's new tokens (see dsa.h)."""
    _call("dsa_pool_compress", ctypes.byref(shape), ctypes.byref(batch), _ptr(cells), _ptr(pos),
          _ptr(pool_keys), _ptr(ws), ws.numel(), _stream(stream))


def dsa_index_prepare(shape, x, pos, rope_dims, rope_base, out, stream=None) -> None:
    """out = H . rope(x, pos), rounded to the shape's dtype (see dsa.h)."""
    _call("dsa_index_prepare", ctypes.byref(shape), int(x.shape[0]), _ptr(x), _ptr(pos),
          int(rope_dims), float(rope_base), _ptr(out), _stream(stream))


def make_pages(page_rows: int, n_pages: int, table_ld: int, fmt=CACHE_E4M3) -> Pages:
    """Geometry of a paged 8-bit cache; ``fmt`` CACHE_E4M3 / CACHE_S8 or "e4m3" / "s8"."""
    fmt = {"e4m3": CACHE_E4M3, "s8": CACHE_S8}.get(fmt, fmt)
    return Pages(int(page_rows), int(fmt), int(n_pages), int(table_ld))


def _refuse(t, dtype, device: int, least: int, what: str):
    if t is None:
        raise ValueError(f"{what} is missing")
    if t.dtype is not dtype:
        raise ValueError(f"{what} is {dtype}, not {t.dtype}")
    if t.numel() < least:
        raise ValueError(f"{what} holds at least {least} elements")
    if not t.is_cuda:
        raise ValueError("libdsa takes CUDA tensors only")
    if t.get_device() != device:
        raise ValueError(f"{what} is on another device than the call's: make its device current")
    raise ValueError("libdsa takes contiguous tensors only")


def _at(t, dtype, device: int, least: int, what: str) -> int:
    """Address of a tensor of the call: its type, size and device are checked."""
    if (t is None or t.dtype is not dtype or t.numel() < least or t.get_device() != device or
            not t.is_contiguous()):
        _refuse(t, dtype, device, least, what)
    return t.data_ptr()


def _bytes_at(t, device: int, count: int, what: str) -> int:
    """Address of a tensor of `count` one-byte elements of any type."""
    if t is None:
        raise ValueError(f"{what} is missing")
    if t.element_size() != 1 or t.numel() != count:
        raise ValueError(f"{what} holds {count} one-byte elements")
    if t.get_device() != device or not t.is_contiguous():
        _refuse(t, t.dtype, device, 0, what)
    return t.data_ptr()


def _count(t, what: str) -> int:
    if t is None:
        raise ValueError(f"{what} is missing")
    return t.numel()


def _stream_at(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def dsa_page_plan(pages, held_len, kv_len, q_len, free_pages, n_free, block_table, row_off, q_off,
                  slots, ws, n_free_out=None, stream=None) -> None:
    """Block tables, slot map (``slots``, one entry per new token) and batch
    offsets from request lengths (see dsa.h); ``n_free_out=None`` updates
    ``n_free`` in place."""
    i64, i32, d = torch.int64, torch.int32, torch.cuda.current_device()
    n, max_new = _count(held_len, "held_len"), _count(slots, "slots")
    free = _at(n_free, i32, d, 1, "n_free")
    _call("dsa_page_plan", pages, n, max_new, _at(held_len, i64, d, n, "held_len"),
          _at(kv_len, i64, d, n, "kv_len"), _at(q_len, i64, d, n, "q_len"),
          _at(free_pages, i32, d, pages.n_pages, "free_pages"), free,
          free if n_free_out is None else _at(n_free_out, i32, d, 1, "n_free_out"),
          _at(block_table, i32, d, n * pages.table_ld, "block_table"),
          _at(row_off, i64, d, n + 1, "row_off"), _at(q_off, i64, d, n + 1, "q_off"),
          _at(slots, i64, d, 0, "slots"), _at(ws, torch.uint8, d, 0, "ws"), ws.numel(),
          _stream_at(stream, d))


def dsa_cache_append(shape, batch, pages, rows, slots, codes, scales, ws, stream=None) -> None:
    """The batch's new rows [n_q, W] rounded into their slots (see dsa.h)."""
    width, d = shape.kv_lora + shape.rope_dim, torch.cuda.current_device()
    n_q, n_pages = batch.n_q, pages.n_pages
    _call("dsa_cache_append", shape, batch, pages,
          _at(rows, _TORCH_DTYPE[shape.dtype], d, n_q * width, "rows"),
          _at(slots, torch.int64, d, n_q, "slots"),
          _bytes_at(codes, d, n_pages * pages.page_rows * width, "codes"),
          _bytes_at(scales, d, n_pages * (2 if shape.rope_dim else 1), "scales"),
          _at(ws, torch.uint8, d, 0, "ws"), ws.numel(), _stream_at(stream, d))


def dsa_paged_mla_attn(shape, batch, pages, q_abs, codes, scales, block_table, idx, n_sel, out,
                       lse, ws, stream=None) -> None:
    """Step 3 over the paged 8-bit cache (see dsa.h)."""
    d, i32, f32 = torch.cuda.current_device(), torch.int32, torch.float32
    n_q, heads, n_pages = batch.n_q, shape.heads, pages.n_pages
    width = shape.kv_lora + shape.rope_dim
    dense = idx is None
    _call("dsa_paged_mla_attn", shape, batch, pages,
          _at(q_abs, _TORCH_DTYPE[shape.dtype], d, n_q * heads * width, "q_abs"),
          _bytes_at(codes, d, n_pages * pages.page_rows * width, "codes"),
          _bytes_at(scales, d, n_pages * (2 if shape.rope_dim else 1), "scales"),
          _at(block_table, i32, d, batch.n_seq * pages.table_ld, "block_table"),
          None if dense else _at(idx, i32, d, n_q * (shape.top_k + shape.kpool - 1), "idx"),
          None if dense else _at(n_sel, i32, d, n_q, "n_sel"),
          _at(out, f32, d, n_q * heads * shape.kv_lora, "out"),
          None if lse is None else _at(lse, f32, d, n_q * heads, "lse"),
          _at(ws, torch.uint8, d, 0, "ws"), ws.numel(), _stream_at(stream, d))


_DSA_DTYPE = {torch.float32: DSA_F32, torch.bfloat16: DSA_BF16}


# The current device, without the look at whether CUDA is there (a tensor of the call is on
# it, or refused): 0.12 of 0.25 us.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _dtype(t, what: str) -> int:
    if t is None:
        raise ValueError(f"{what} is missing")
    d = _DSA_DTYPE.get(t.dtype)
    if d is None:
        raise ValueError(f"{what} is float32 or bfloat16, not {t.dtype}")
    return d


def _rows_at(t, like, dtype, device: int, what: str):
    """Address and row stride of a matrix of ``like``'s shape whose rows may be
    parts of wider ones."""
    if t is None:
        raise ValueError(f"{what} is missing")
    if t.shape != like or t.dtype is not dtype or t.get_device() != device:
        if t.shape != like:
            raise ValueError(f"{what} has the shape {tuple(like)}, not {tuple(t.shape)}")
        _refuse(t, dtype, device, 0, what)
    ld, step = t.stride()
    rows, width = like
    if step != 1 and width > 1:
        raise ValueError(f"{what}'s rows are contiguous: its last stride is 1")
    return t.data_ptr(), ld if rows > 1 else width


# Types that an output of e4m3 codes may have; others of one byte would be read as other numbers.
_CODES = (torch.float8_e4m3fn, torch.uint8)


def dsa_rms_norm(x, weight, eps, out, add=None, total=None, scales=None, group=0,
                 stream=None) -> None:
    """Norm of the rows of ``x`` [rows, width], or of ``x + add`` (see dsa.h);
    ``total`` gets the sum.  ``out`` has x's type, or is float8_e4m3fn or uint8 (e4m3
    codes) with ``scales`` [rows, ceil(width / group)] float32 (group 0: [rows, 1])."""
    kind, d = _dtype(x, "x"), _device()
    like, dt = x.shape, x.dtype
    if len(like) != 2:
        raise ValueError("x is a matrix of rows")
    rows, width = like
    px, x_ld = _rows_at(x, like, dt, d, "x")
    pa, a_ld = (None, 0) if add is None else _rows_at(add, like, dt, d, "add")
    pt, t_ld = (None, 0) if total is None else _rows_at(total, like, dt, d, "total")
    codes = out is not None and out.dtype in _CODES
    po, o_ld = _rows_at(out, like, out.dtype if codes else dt, d, "out")
    ps = None
    if codes:
        ps = _at(scales, torch.float32, d, rows * (-(-width // group) if group else 1), "scales")
    elif scales is not None:
        raise ValueError("scales go with an out of float8_e4m3fn or uint8")
    _call("dsa_rms_norm", rows, width, kind, px, x_ld, pa, a_ld,
          None if weight is None else _at(weight, torch.float32, d, width, "weight"), eps, pt, t_ld, po,
          o_ld, NORM_E4M3 if codes else NORM_SAME, ps, group, _stream_at(stream, d))


def dsa_rope_init(plan, dims, layout=ROPE_PAIRS, inverse=0, base=8e6, factor=1.0, original_len=0.0,
                  beta_fast=32.0, beta_slow=1.0, magnitude=1.0) -> None:
    """Fills a :class:`RopePlan` (see dsa.h)."""
    _call("dsa_rope_init", ctypes.byref(plan), int(dims), int(layout), int(inverse), base, factor,
          original_len, beta_fast, beta_slow, magnitude)


def make_rope(dims, base, layout="pairs", factor=1.0, original_len=0.0, beta_fast=32.0,
              beta_slow=1.0, magnitude=1.0, inverse=False) -> RopePlan:
    """Plan of ``dsa_rope``: ``layout`` ROPE_PAIRS / ROPE_HALVES or "pairs" / "halves"."""
    plan = RopePlan()
    layout = {"pairs": ROPE_PAIRS, "halves": ROPE_HALVES}.get(layout, layout)
    dsa_rope_init(plan, dims, layout, inverse, base, factor, original_len, beta_fast, beta_slow, magnitude)
    return plan


def _heads_at(t, like, dtype, device: int, what: str):
    """Address and the strides of tokens and heads of [tokens, heads, dims] or
    [tokens, dims], the last dimension contiguous."""
    if t is None:
        raise ValueError(f"{what} is missing")
    if t.shape != like or t.dtype is not dtype or t.get_device() != device:
        if t.shape != like:
            raise ValueError(f"{what} has the shape {tuple(like)}, not {tuple(t.shape)}")
        _refuse(t, dtype, device, 0, what)
    s = t.stride()
    if s[-1] != 1:
        raise ValueError(f"{what}'s heads are contiguous: its last stride is 1")
    return t.data_ptr(), s[0], s[1] if len(s) == 3 else 0


def dsa_rope(rope, x, pos, out, stream=None) -> None:
    """``x`` [tokens, heads, dims] or [tokens, dims] (views of the rotated columns)
    turned by ``pos`` [tokens] int64 into ``out``, which may be x (see dsa.h)."""
    kind, d = _dtype(x, "x"), _device()
    like, dt = x.shape, x.dtype
    if len(like) not in (2, 3) or like[-1] != rope.dims:
        raise ValueError(f"x is [tokens, heads, {rope.dims}] or [tokens, {rope.dims}]")
    tokens = like[0]
    px, x_tok, x_head = _heads_at(x, like, dt, d, "x")
    po, o_tok, o_head = _heads_at(out, like, dt, d, "out")
    _call("dsa_rope", rope, kind, tokens, like[1] if len(like) == 3 else 1, px, x_tok, x_head,
          _at(pos, torch.int64, d, tokens, "pos"), po, o_tok, o_head, _stream_at(stream, d))


def _weights_at(t, shape, device: int, what: str):
    """Address and middle size of a weight [heads, features, kv_lora]."""
    if t is None:
        raise ValueError(f"{what} is missing")
    n = t.shape[1] if t.dim() == 3 else 0
    if t.dim() != 3 or t.shape[0] != shape.heads or t.shape[2] != shape.kv_lora:
        raise ValueError(f"{what} is [{shape.heads}, features, {shape.kv_lora}]")
    return _at(t, _TORCH_DTYPE[shape.dtype], device, 0, what), n


def dsa_expand_kv(shape, cache, w_uk, w_uv, k_nope, v, ws, stream=None) -> None:
    """``cache`` [rows, W] expanded into ``k_nope`` [rows, heads, nope] and ``v``
    [rows, heads, v_dim] (see dsa.h)."""
    d, dt = _device(), _TORCH_DTYPE[shape.dtype]
    pk, nope = _weights_at(w_uk, shape, d, "w_uk")
    pv, v_dim = _weights_at(w_uv, shape, d, "w_uv")
    if cache is None or cache.dim() != 2 or cache.shape[1] != shape.kv_lora + shape.rope_dim:
        raise ValueError(f"cache is [rows, {shape.kv_lora + shape.rope_dim}]")
    rows = cache.shape[0]
    _call("dsa_expand_kv", shape, rows, nope, v_dim, _at(cache, dt, d, 0, "cache"), pk, pv,
          _at(k_nope, dt, d, rows * shape.heads * nope, "k_nope"),
          _at(v, dt, d, rows * shape.heads * v_dim, "v"), _at(ws, torch.uint8, d, 0, "ws"), ws.numel(),
          _stream_at(stream, d))


def dsa_expanded_mla_attn(shape, batch, q, k_nope, cache, v, out, lse, ws, stream=None) -> None:
    """Causal attention over expanded keys ``k_nope`` [rows, heads, nope] and values
    ``v`` [rows, heads, v_dim], the rope part of the keys in ``cache`` (see dsa.h)."""
    d, dt = _device(), _TORCH_DTYPE[shape.dtype]
    heads, rope, n_q, rows = shape.heads, shape.rope_dim, batch.n_q, batch.total_rows
    if k_nope is None or v is None or k_nope.dim() != 3 or v.dim() != 3 or \
            k_nope.shape[1] != heads or v.shape[1] != heads:
        raise ValueError(f"k_nope and v are [rows, {heads}, columns]")
    nope, v_dim = k_nope.shape[2], v.shape[2]
    _call("dsa_expanded_mla_attn", shape, batch, nope, v_dim,
          _at(q, dt, d, n_q * heads * (nope + rope), "q"),
          _at(k_nope, dt, d, rows * heads * nope, "k_nope"),
          _at(cache, dt, d, rows * (shape.kv_lora + rope), "cache") if rope else None,
          _at(v, dt, d, rows * heads * v_dim, "v"), _at(out, dt, d, n_q * heads * v_dim, "out"),
          None if lse is None else _at(lse, torch.float32, d, n_q * heads, "lse"),
          _at(ws, torch.uint8, d, 0, "ws"), ws.numel(), _stream_at(stream, d))


def dsa_check_device_error(ws: Optional[torch.Tensor], stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error code;
    ``ws=None`` reads the no-allocation entry point's scratch array."""
    code = ctypes.c_int32(0)
    rc = load().dsa_check_device_error(_ptr(ws), ws.numel() if ws is not None else 0,
                                       _stream(stream), ctypes.byref(code))
    if rc not in (0, 5, 6):
        raise DsaError("dsa_check_device_error", rc)
    return int(code.value)


def dsa_absorb_q(shape, q, w_uk, q_abs, ws, stream=None) -> None:
    """q [n_q, heads, nope + rope], w_uk [heads, nope, kv_lora] -> q_abs (see dsa.h)."""
    _call("dsa_absorb_q", ctypes.byref(shape), int(q.shape[0]), int(w_uk.shape[1]), _ptr(q),
          _ptr(w_uk), _ptr(q_abs), _ptr(ws), ws.numel(), _stream(stream))


def dsa_up_project(shape, o, w_uv, out, ws, stream=None) -> None:
    """o [n_q, heads, kv_lora] float32, w_uv [heads, v_dim, kv_lora] -> out (see dsa.h)."""
    _call("dsa_up_project", ctypes.byref(shape), int(o.shape[0]), int(w_uv.shape[1]), _ptr(o),
          _ptr(w_uv), _ptr(out), _ptr(ws), ws.numel(), _stream(stream))


def dsa_workspace_set_wait_budget(ws: torch.Tensor, ns: int, stream=None) -> None:
    """Budget of the waits between CTAs of kernels using ``ws`` (0 = default)."""
    _call("dsa_workspace_set_wait_budget", _ptr(ws), ws.numel(), int(ns), _stream(stream))


class DecodeStep:
    """The whole hot path for a fixed batch layout, with its own workspace.

    ``inputs`` is a dict with the tensors of the layout above plus the int64
    offset arrays ``row_off``, ``key_off``, ``q_off`` (all on one CUDA device);
    ``wl`` supplies the geometry (``top_k``, ``kpool``, ``rope``, ``scale``,
    ``dtype``, ``kv_lens``, ``q_lens``).
    """

    def __init__(self, wl, row_off, key_off, q_off, device="cuda"):
        self.shape = make_shape(wl.idx_heads, wl.idx_dim, wl.heads, wl.kv_lora, wl.rope, wl.top_k,
                                wl.kpool, wl.scale, wl.dtype)
        self.batch = make_batch(row_off, key_off, q_off, wl.n_q, max(wl.q_lens), max(wl.kv_lens),
                                sum(wl.kv_lens), sum(wl.key_counts()))
        self.ws = alloc_workspace(self.shape, self.batch, OP_DECODE_STEP, device)
        self.width = dsa_index_row_width(self.shape)
        self.n_q = wl.n_q
        self.heads, self.kv_lora = wl.heads, wl.kv_lora
        dev = self.ws.device
        self.idx = torch.empty((self.n_q, self.width), dtype=torch.int32, device=dev)
        self.n_sel = torch.empty(self.n_q, dtype=torch.int32, device=dev)

    def __call__(self, q_idx, w, k_idx, q_abs, cache, out, lse=None, stream=None):
        dsa_decode_step(self.shape, self.batch, q_idx, w, k_idx, q_abs, cache, out, lse,
                        self.idx, self.n_sel, self.ws, stream)
