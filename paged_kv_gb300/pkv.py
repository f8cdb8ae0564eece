"""Thin binding of ``libpkv.so`` (the C ABI in ``include/pkv.h``): by ctypes, and for
the serving operators by ``_binding.so`` (``csrc/binding.cpp``).

Argument marshalling only: every step of the sampler, the write-back and the
page fill runs in the library's CUDA kernels.  PyTorch supplies device memory
and the current stream.  The functions keep the C names without the ``pkv_``
prefix and raise ``PkvError`` on a negative status.  There is no CPU fallback:
if ``libpkv.so`` has not been built (``__graft_entry__.build()``) every call
raises.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK, PKV_EINVAL, PKV_ENOSPC, PKV_ECUDA, PKV_EUNSUPPORTED = 0, -1, -2, -3, -4
PKV_FP32, PKV_BF16, PKV_FP16 = 0, 1, 2
PKV_MAX_VOCAB_FP32, PKV_MAX_VOCAB_BF16 = 262144, 524288
PKV_MAX_HEAD_DIM = 128
PKV_ATTENTION_ZERO_BYTES = 65536
ST_NONFINITE, ST_ALL_NEG_INF, ST_ROW_OOB, ST_COL_OOB, ST_BAD_UNIFORM, ST_NOSPC = 1, 2, 4, 8, 16, 32
ST_TIMEOUT = 64
ST_TOKEN_CAP = 128
FL_COUNT, FL_ALIGN, FL_RANGE, FL_DUPLICATE = 1, 2, 4, 8

_lock = threading.Lock()
_lib = None


class PkvError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"pkv error {code}: {message}")
        self.code = code


def load() -> ctypes.CDLL:
    """Load libpkv.so (raises if it is missing: there is no fallback path)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            lib = ctypes.CDLL(LIB_PATH)
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            lib.pkv_last_error.restype = ctypes.c_char_p
            lib.pkv_last_error.argtypes = []
            lib.pkv_version.restype = i32
            lib.pkv_version.argtypes = []
            lib.pkv_sample_workspace_bytes.restype = sz
            lib.pkv_sample_workspace_bytes.argtypes = [i32, i32, i32]
            lib.pkv_sample_batch_noalloc.restype = i32
            lib.pkv_sample_batch_noalloc.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp,
                                                     vp, i64, i64, vp, vp, vp, vp, vp]
            lib.pkv_decode_tail.restype = i32
            lib.pkv_decode_tail.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, i64,
                                            i64, vp, vp, vp, vp, sz, vp, vp, vp, i32, i32, vp,
                                            i64, vp, i64, i64, vp, vp]
            lib.pkv_sample_workspace_init.restype = i32
            lib.pkv_sample_workspace_init.argtypes = [vp, sz, vp]
            lib.pkv_sample_batch_ex.restype = i32
            lib.pkv_sample_batch_ex.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp,
                                                vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]
            lib.pkv_sample_batch.restype = i32
            lib.pkv_sample_batch.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp,
                                             i64, i64, vp, vp, vp, vp, vp, sz, vp]
            lib.pkv_writeback_tokens.restype = i32
            lib.pkv_writeback_tokens.argtypes = [vp, vp, vp, i32, vp, i64, i64, vp, vp]
            lib.pkv_alloc_pages.restype = i32
            lib.pkv_alloc_pages.argtypes = [vp, vp, i32, i32, i64, vp, vp, vp, vp]
            lib.pkv_fill_page_table.restype = i32
            lib.pkv_fill_page_table.argtypes = [vp, vp, vp, i32, i32, vp, i64, vp, i64, i64,
                                                vp, vp, vp]
            lib.pkv_free_pages.restype = i32
            lib.pkv_free_pages.argtypes = [vp, vp, vp, i32, i32, vp, i64, i64, vp, i64, i64,
                                           vp, vp, vp]
            lib.pkv_prepare_step.restype = i32
            lib.pkv_prepare_step.argtypes = [vp, vp, vp, i32, i32, vp, i64, vp, i64, i64, vp,
                                             i64, i64, vp, vp, vp, i64, vp, vp, vp, vp]
            lib.pkv_philox_uniforms.restype = i32
            lib.pkv_philox_uniforms.argtypes = [ctypes.c_uint64, ctypes.c_uint64, i32, vp, vp]
            f32 = ctypes.c_float
            lib.pkv_append_kv.restype = i32
            lib.pkv_append_kv.argtypes = [vp, vp, i64, i64, vp, i64, i64, i32, i64, vp, vp, vp, vp,
                                          i64, i32, i32, vp, i64, i64, i32, vp, i64, i64, vp, vp]
            lib.pkv_paged_attention_workspace_bytes.restype = sz
            lib.pkv_paged_attention_workspace_bytes.argtypes = [i32, i64, i32, i32, i32, i32]
            lib.pkv_paged_attention.restype = i32
            lib.pkv_paged_attention.argtypes = [vp, vp, i64, i64, i32, i32, i64, vp, i64, i64, vp,
                                                vp, vp, vp, vp, i32, i32, vp, i64, i64, f32, i32,
                                                vp, vp, sz, vp]
            lib.pkv_adjust_logits.restype = i32
            lib.pkv_adjust_logits.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, i64, i64, vp,
                                              vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64, vp, vp]
            lib.pkv_check_free_list.restype = i32
            lib.pkv_check_free_list.argtypes = [vp, i64, i32, i64, i64, vp, i64, vp, vp]
            _lib = lib
    return _lib


def last_error() -> str:
    return load().pkv_last_error().decode()


def version() -> int:
    return load().pkv_version()


def _check(rc: int) -> None:
    if rc != PKV_OK:
        raise PkvError(rc, last_error())


def _dev(t: Optional[torch.Tensor], dtype: torch.dtype, name: str, n: Optional[int] = None):
    """Device pointer of a contiguous CUDA tensor of the given dtype (or None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if n is not None and t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, needs {n}")
    return t.data_ptr()


def _stream(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_workspaces = {}


def sample_workspace_bytes(B: int, V: int, dtype: torch.dtype) -> int:
    """pkv_sample_workspace_bytes for a [B, V] batch of ``dtype`` logits."""
    code = PKV_BF16 if dtype == torch.bfloat16 else PKV_FP32
    return int(load().pkv_sample_workspace_bytes(int(B), int(V), code))


def sample_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    """pkv_sample_workspace_init: readies a new workspace (zeroes its header)."""
    if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 CUDA tensor")
    _check(load().pkv_sample_workspace_init(workspace.data_ptr(), workspace.numel(),
                                            _stream(stream, workspace.device)))


def _workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    """A cached, zero-initialised uint8 device buffer of at least ``nbytes``
    (replaced by a larger one as needed).

    Calls on different streams of one device must pass their own workspace.
    """
    key = (device.type, device.index)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def sample_batch(logits: torch.Tensor, temperature: Optional[torch.Tensor] = None,
                 top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
                 uniform: Optional[torch.Tensor] = None,
                 out_tokens: Optional[torch.Tensor] = None,
                 token_pool: Optional[torch.Tensor] = None,
                 wb_rows: Optional[torch.Tensor] = None, wb_cols: Optional[torch.Tensor] = None,
                 probs_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None,
                 min_p: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pkv_sample_batch: one int32 token per row of ``logits`` [B, V]
    (pkv_sample_batch_ex when ``min_p`` is given).

    ``logits`` is fp32 or bf16 with unit column stride (any row stride).
    ``workspace`` (a uint8 CUDA tensor, initialised once with
    sample_workspace_init or zeroed) defaults to a buffer cached per device.
    Returns ``out_tokens`` (allocated here if not given).  See include/pkv.h.
    """
    lib = load()
    if logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a 2-D CUDA tensor")
    if logits.stride(1) != 1:
        raise ValueError("logits must have unit column stride")
    if logits.dtype == torch.bfloat16:
        dcode = PKV_BF16
    elif logits.dtype == torch.float32:
        dcode = PKV_FP32
    else:
        raise TypeError(f"logits dtype {logits.dtype} is not fp32 or bf16")
    B, V = logits.shape
    if out_tokens is None:
        out_tokens = torch.empty(B, dtype=torch.int32, device=logits.device)
    pool_rows = pool_cols = 0
    if token_pool is not None:
        if token_pool.dim() != 2:
            raise ValueError("token_pool must be 2-D")
        pool_rows, pool_cols = token_pool.shape
    need = int(lib.pkv_sample_workspace_bytes(B, V, dcode))
    if workspace is None:
        workspace = _workspace(logits.device, need)
    if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 CUDA tensor")
    head = (logits.data_ptr(), dcode, B, V, logits.stride(0),
            _dev(temperature, torch.float32, "temperature", B),
            _dev(top_k, torch.int32, "top_k", B), _dev(top_p, torch.float32, "top_p", B))
    if min_p is not None:
        call = lambda *rest: lib.pkv_sample_batch_ex(  # noqa: E731
            *head, _dev(min_p, torch.float32, "min_p", B), *rest)
    else:
        call = lambda *rest: lib.pkv_sample_batch(*head, *rest)  # noqa: E731
    rc = call(
        _dev(uniform, torch.float32, "uniform", B), _dev(out_tokens, torch.int32, "out_tokens", B),
        _dev(token_pool, torch.int32, "token_pool"), pool_rows, pool_cols,
        _dev(wb_rows, torch.int32, "wb_rows", B), _dev(wb_cols, torch.int64, "wb_cols", B),
        _dev(probs_out, torch.float32, "probs_out", B * V), _dev(status, torch.int32, "status", 1),
        workspace.data_ptr(), workspace.numel(), _stream(stream, logits.device))
    _check(rc)
    return out_tokens


def sample_batch_noalloc(logits: torch.Tensor, temperature: Optional[torch.Tensor] = None,
                         top_k: Optional[torch.Tensor] = None,
                         top_p: Optional[torch.Tensor] = None,
                         uniform: Optional[torch.Tensor] = None,
                         out_tokens: torch.Tensor = None,
                         token_pool: Optional[torch.Tensor] = None,
                         wb_rows: Optional[torch.Tensor] = None,
                         wb_cols: Optional[torch.Tensor] = None,
                         probs_out: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_sample_batch_noalloc: sample_batch with the library's own static
    scratch; ``out_tokens`` (int32 [B], on the logits' device) is required, so
    that nothing is allocated.  See include/pkv.h."""
    lib = load()
    if logits.dim() != 2 or not logits.is_cuda or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D CUDA tensor with unit column stride")
    if logits.dtype == torch.bfloat16:
        dcode = PKV_BF16
    elif logits.dtype == torch.float32:
        dcode = PKV_FP32
    else:
        raise TypeError(f"logits dtype {logits.dtype} is not fp32 or bf16")
    if out_tokens is None:
        raise ValueError("out_tokens is required")
    B, V = logits.shape
    pool_rows = pool_cols = 0
    if token_pool is not None:
        if token_pool.dim() != 2:
            raise ValueError("token_pool must be 2-D")
        pool_rows, pool_cols = token_pool.shape
    rc = lib.pkv_sample_batch_noalloc(
        logits.data_ptr(), dcode, B, V, logits.stride(0),
        _dev(temperature, torch.float32, "temperature", B),
        _dev(top_k, torch.int32, "top_k", B), _dev(top_p, torch.float32, "top_p", B),
        _dev(uniform, torch.float32, "uniform", B), _dev(out_tokens, torch.int32, "out_tokens", B),
        _dev(token_pool, torch.int32, "token_pool"), pool_rows, pool_cols,
        _dev(wb_rows, torch.int32, "wb_rows", B), _dev(wb_cols, torch.int64, "wb_cols", B),
        _dev(probs_out, torch.float32, "probs_out", B * V), _dev(status, torch.int32, "status", 1),
        _stream(stream, logits.device))
    _check(rc)
    return out_tokens


def decode_tail(logits: torch.Tensor, temperature, top_k, top_p, uniform,
                out_tokens: torch.Tensor, token_pool, wb_rows, wb_cols,
                cached_len: torch.Tensor, device_len: torch.Tensor, table_idx: torch.Tensor,
                page_size: int, free_slots: torch.Tensor, page_table: torch.Tensor,
                total_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_decode_tail: sample_batch (with its write-back) and fill_page_table
    of one decode step in one call.  Returns ``out_tokens``."""
    lib = load()
    if logits.dim() != 2 or not logits.is_cuda or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D CUDA tensor with unit column stride")
    if logits.dtype == torch.bfloat16:
        dcode = PKV_BF16
    elif logits.dtype == torch.float32:
        dcode = PKV_FP32
    else:
        raise TypeError(f"logits dtype {logits.dtype} is not fp32 or bf16")
    B, V = logits.shape
    pool_rows = pool_cols = 0
    if token_pool is not None:
        pool_rows, pool_cols = token_pool.shape
    if page_table.dim() != 2:
        raise ValueError("page_table must be 2-D")
    need = int(lib.pkv_sample_workspace_bytes(B, V, dcode))
    if workspace is None:
        workspace = _workspace(logits.device, need)
    fb = cached_len.numel()
    rc = lib.pkv_decode_tail(
        logits.data_ptr(), dcode, B, V, logits.stride(0),
        _dev(temperature, torch.float32, "temperature", B),
        _dev(top_k, torch.int32, "top_k", B), _dev(top_p, torch.float32, "top_p", B),
        _dev(uniform, torch.float32, "uniform", B), _dev(out_tokens, torch.int32, "out_tokens", B),
        _dev(token_pool, torch.int32, "token_pool"), pool_rows, pool_cols,
        _dev(wb_rows, torch.int32, "wb_rows", B), _dev(wb_cols, torch.int64, "wb_cols", B),
        _dev(status, torch.int32, "status", 1), workspace.data_ptr(), workspace.numel(),
        _dev(cached_len, torch.int32, "cached_len", fb),
        _dev(device_len, torch.int32, "device_len", fb),
        _dev(table_idx, torch.int32, "table_idx", fb), fb, int(page_size),
        _dev(free_slots, torch.int32, "free_slots"), free_slots.numel(),
        _dev(page_table, torch.int32, "page_table"), page_table.shape[0], page_table.shape[1],
        _dev(total_out, torch.int64, "total_out", 1), _stream(stream, logits.device))
    _check(rc)
    return out_tokens


def writeback_tokens(tokens: torch.Tensor, rows: torch.Tensor, cols: torch.Tensor,
                     token_pool: torch.Tensor, status: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """pkv_writeback_tokens: token_pool[rows[b], cols[b]] = tokens[b] (cols < 0 skipped)."""
    lib = load()
    B = tokens.numel()
    R, C = token_pool.shape
    rc = lib.pkv_writeback_tokens(
        _dev(tokens, torch.int32, "tokens"), _dev(rows, torch.int32, "rows", B),
        _dev(cols, torch.int64, "cols", B), B, _dev(token_pool, torch.int32, "token_pool"),
        R, C, _dev(status, torch.int32, "status", 1), _stream(stream, token_pool.device))
    _check(rc)


def alloc_pages(cached_len, device_len, page_size: int, free_count: int) -> dict:
    """pkv_alloc_pages on host int32 arrays; returns first_page, num_pages, offset, total.

    Raises PkvError(PKV_ENOSPC) when the total exceeds free_count.
    """
    lib = load()
    c = torch.as_tensor(cached_len, dtype=torch.int32).contiguous().cpu()
    d = torch.as_tensor(device_len, dtype=torch.int32).contiguous().cpu()
    B = c.numel()
    first = torch.empty(B, dtype=torch.int32)
    num = torch.empty(B, dtype=torch.int32)
    off = torch.empty(B, dtype=torch.int64)
    total = torch.zeros(1, dtype=torch.int64)
    rc = lib.pkv_alloc_pages(c.data_ptr(), d.data_ptr(), B, int(page_size), int(free_count),
                             first.data_ptr(), num.data_ptr(), off.data_ptr(), total.data_ptr())
    out = {"first_page": first, "num_pages": num, "offset": off, "total": int(total[0])}
    _check(rc)
    return out


def fill_page_table(cached_len: torch.Tensor, device_len: torch.Tensor, table_idx: torch.Tensor,
                    page_size: int, free_slots: torch.Tensor, page_table: torch.Tensor,
                    total_out: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """pkv_fill_page_table: allocate from the front of ``free_slots`` and fill ``page_table``."""
    lib = load()
    B = cached_len.numel()
    R, C = page_table.shape
    rc = lib.pkv_fill_page_table(
        _dev(cached_len, torch.int32, "cached_len", B), _dev(device_len, torch.int32, "device_len", B),
        _dev(table_idx, torch.int32, "table_idx", B), B, int(page_size),
        _dev(free_slots, torch.int32, "free_slots"), free_slots.numel(),
        _dev(page_table, torch.int32, "page_table"), R, C,
        _dev(total_out, torch.int64, "total_out", 1), _dev(status, torch.int32, "status", 1),
        _stream(stream, page_table.device))
    _check(rc)


def prepare_step(cached_len: torch.Tensor, device_len: torch.Tensor, table_idx: torch.Tensor,
                 page_size: int, free_slots: torch.Tensor, page_table: torch.Tensor,
                 token_pool: torch.Tensor, max_tokens: int,
                 positions: Optional[torch.Tensor] = None,
                 input_ids: Optional[torch.Tensor] = None,
                 out_loc: Optional[torch.Tensor] = None,
                 total_pages: Optional[torch.Tensor] = None,
                 total_tokens: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None):
    """pkv_prepare_step: allocate and fill this step's pages, pack the
    positions [cached_len, device_len) and gather input_ids / out_loc at
    (table_idx, position).  Returns (positions, input_ids, out_loc,
    total_pages, total_tokens) as device tensors; the first three hold
    ``max_tokens`` entries, of which the first total_tokens are the step's."""
    lib = load()
    B = cached_len.numel()
    dev = page_table.device
    R, C = page_table.shape
    PR, PC = token_pool.shape
    n = int(max_tokens)

    def out(t, dtype, k):
        return t if t is not None else torch.empty(k, dtype=dtype, device=dev)

    positions = out(positions, torch.int32, n)
    input_ids = out(input_ids, torch.int32, n)
    out_loc = out(out_loc, torch.int32, n)
    total_pages = out(total_pages, torch.int64, 1)
    total_tokens = out(total_tokens, torch.int64, 1)
    rc = lib.pkv_prepare_step(
        _dev(cached_len, torch.int32, "cached_len", B), _dev(device_len, torch.int32, "device_len", B),
        _dev(table_idx, torch.int32, "table_idx", B), B, int(page_size),
        _dev(free_slots, torch.int32, "free_slots"), free_slots.numel(),
        _dev(page_table, torch.int32, "page_table"), R, C,
        _dev(token_pool, torch.int32, "token_pool"), PR, PC,
        _dev(positions, torch.int32, "positions", n), _dev(input_ids, torch.int32, "input_ids", n),
        _dev(out_loc, torch.int32, "out_loc", n), n,
        _dev(total_pages, torch.int64, "total_pages", 1),
        _dev(total_tokens, torch.int64, "total_tokens", 1),
        _dev(status, torch.int32, "status", 1), _stream(stream, dev))
    _check(rc)
    return positions, input_ids, out_loc, total_pages, total_tokens


def philox_uniforms(seed: int, offset: int, B: int, out: Optional[torch.Tensor] = None,
                    device=None, stream=None) -> torch.Tensor:
    """pkv_philox_uniforms: the B float32 uniforms of call ``offset`` under
    ``seed``, generated on the device."""
    if out is None:
        out = torch.empty(int(B), dtype=torch.float32,
                          device=device if device is not None else "cuda")
    rc = load().pkv_philox_uniforms(int(seed) & ((1 << 64) - 1), int(offset) & ((1 << 64) - 1),
                                    int(B), _dev(out, torch.float32, "out", int(B)),
                                    _stream(stream, out.device))
    _check(rc)
    return out


def free_pages(table_idx: torch.Tensor, begin: torch.Tensor, end: torch.Tensor, page_size: int,
               page_table: torch.Tensor, free_slots: torch.Tensor, free_count: int,
               total_out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None) -> None:
    """pkv_free_pages: append page_table[t, b:e:ps] of every request after the
    ``free_count`` live entries of ``free_slots`` (whose length is the capacity)."""
    lib = load()
    B = table_idx.numel()
    R, C = page_table.shape
    rc = lib.pkv_free_pages(
        _dev(table_idx, torch.int32, "table_idx", B), _dev(begin, torch.int32, "begin", B),
        _dev(end, torch.int32, "end", B), B, int(page_size),
        _dev(page_table, torch.int32, "page_table"), R, C,
        _dev(free_slots, torch.int32, "free_slots"), int(free_count), free_slots.numel(),
        _dev(total_out, torch.int64, "total_out", 1), _dev(status, torch.int32, "status", 1),
        _stream(stream, page_table.device))
    _check(rc)


def check_free_list(free_slots: torch.Tensor, free_count: int, page_size: int, num_pages: int,
                    cache_pages: int, bitmap: torch.Tensor, result: torch.Tensor,
                    stream=None) -> None:
    """pkv_check_free_list: OR the FL_* bits of the first ``free_count`` entries
    into ``result`` (zeroed first); ``bitmap`` is int32 scratch of
    ceil(num_pages / 32) words."""
    lib = load()
    rc = lib.pkv_check_free_list(
        _dev(free_slots, torch.int32, "free_slots"), int(free_count), int(page_size),
        int(num_pages), int(cache_pages), _dev(bitmap, torch.int32, "bitmap"), bitmap.numel(),
        _dev(result, torch.int32, "result", 1), _stream(stream, result.device))
    _check(rc)


# ------------------------------------------------------------------ the paged KV cache


class _KVCacheStruct(ctypes.Structure):
    """pkv_kv_cache of include/pkv.h."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class KVCache:
    """One layer's paged keys and values in 8 bits (pkv_kv_cache).

    ``k`` and ``v`` are float8_e4m3fn [num_pages, page_size, kv_heads, head_dim]
    with the same strides, the last of them 1 and the others multiples of 16;
    ``k_scale`` and ``v_scale`` are contiguous fp32 [num_pages, kv_heads].  The
    object keeps the tensors alive; it is made once and passed to every call.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a CUDA tensor")
            if t.dtype != torch.float8_e4m3fn:
                raise TypeError(f"{name} must be torch.float8_e4m3fn, got {t.dtype}")
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{name} must be [pages, page_size, kv_heads, head_dim] with unit "
                                 "last stride")
        pages, ps, heads, dim = k.shape
        # The stride of a dimension of one is never used, and torch leaves any value in it.
        strides, v_strides = ([x.stride(i) if x.shape[i] > 1 else 0 for i in range(3)]
                              for x in (k, v))
        if k.shape != v.shape or strides != v_strides or k.device != v.device:
            raise ValueError("k and v must have the same shape, strides and device")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _dev(t, torch.float32, name, pages * heads)
            if tuple(t.shape) != (pages, heads) or t.device != k.device:
                raise ValueError(f"{name} must be [{pages}, {heads}] on {k.device}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = pages, ps, heads, dim
        self.device = k.device
        self._struct = _KVCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                      v_scale.data_ptr(), pages, *strides, ps, heads, dim, 0)
        self._ref = ctypes.addressof(self._struct)
        self._index = k.device.index

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
              device="cuda") -> "KVCache":
        """A new cache (codes zero, scales one) in which a page's tokens lie next
        to one another for each head, so that attention reads whole pages in one
        piece."""
        shape = (int(num_pages), int(kv_heads), int(page_size), int(head_dim))

        def codes():
            t = torch.zeros(shape, dtype=torch.uint8, device=device)
            return t.view(torch.float8_e4m3fn).permute(0, 2, 1, 3)

        def scales():
            return torch.ones(shape[:2], dtype=torch.float32, device=device)

        return cls(codes(), codes(), scales(), scales())


_binding = None


def _bind():
    """The compiled binding of the serving operators (paged_kv_gb300/_binding.so)."""
    global _binding
    if _binding is None:
        load()
        from . import _binding as module

        _binding = module
    return _binding


def _torch_stream(stream, device):
    """A stream object or handle as one of torch's."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream(stream, device)
    # (1 and 2 name the legacy and the calling thread's default stream.)
    return (torch.cuda.ExternalStream(handle, device=device) if handle > 2
            else torch.cuda.default_stream(device))


def _new_like(q: torch.Tensor, stream) -> torch.Tensor:
    """A dense output of ``q``'s shape, in memory of the call's stream: another stream's
    may still be written there by work that came before."""
    if stream is None or not q.is_cuda:  # (the binding refuses the latter)
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)
    with torch.cuda.stream(_torch_stream(stream, q.device)):
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)


def append_kv(cache: KVCache, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
              out_loc: torch.Tensor, cos_sin: Optional[torch.Tensor] = None,
              interleaved: bool = False, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, total_tokens: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """pkv_append_kv: write the packed tokens' ``k`` and ``v`` [n, kv_heads, head_dim]
    into ``cache`` at ``out_loc``, with k and ``q`` [n, q_heads, head_dim] rotated by
    ``positions`` under ``cos_sin`` [max_pos, rot_dim] (cosines, then sines; None: no
    rotation).  Returns the rotated queries (``q_out``, allocated here if not given;
    None without ``q``).  See include/pkv.h."""
    if q is not None and q_out is None:
        q_out = _new_like(q, stream)
    rc = (_binding or _bind()).append_kv(cache._ref, cache._index, k, v, positions, out_loc, cos_sin,
                                         interleaved, q, q_out, total_tokens, status, stream)
    if rc:
        _check(rc)
    return q_out


# Default workspaces, by stream handle and device: made once, never replaced or dropped,
# so that a call in flight keeps its own.  Those of captures, with the capture's id.
_attention_workspaces = {}
_capture_workspaces = {}


def _default_attention_workspace(need, handle, key, capture, index) -> torch.Tensor:
    """The workspace of the calls on one stream, made and zeroed on that stream.

    A stream that is being captured gets one of the capture's: it lies in the graph's
    memory and each replay zeroes it, so neither other graphs nor calls outside share
    it.  It is kept for the capture's later calls.
    """
    if capture == 0:
        # The most that any call of this device needs.
        need = paged_attention_workspace_bytes(1, 64, 64, 1, 1, PKV_MAX_HEAD_DIM)
    with _lock:
        if capture == 0:
            ws = _attention_workspaces.get(key)
        else:
            owner, ws = _capture_workspaces.get(key, (0, None))
            if owner != capture or ws.numel() < need:
                ws = None
        if ws is None:
            device = torch.device("cuda", index)
            with torch.cuda.stream(_torch_stream(handle, device)):
                ws = torch.empty(need, dtype=torch.uint8, device=device)
                ws[:PKV_ATTENTION_ZERO_BYTES].zero_()
            if capture == 0:
                _attention_workspaces[key] = ws
            else:
                _capture_workspaces[key] = (capture, ws)
    return ws


def paged_attention_workspace_bytes(B: int, n_tokens: int, max_q_len: int, q_heads: int,
                                    kv_heads: int, head_dim: int) -> int:
    """pkv_paged_attention_workspace_bytes."""
    return int(load().pkv_paged_attention_workspace_bytes(int(B), int(n_tokens), int(max_q_len),
                                                          int(q_heads), int(kv_heads),
                                                          int(head_dim)))


def paged_attention(q: torch.Tensor, cache: KVCache, cached_len: torch.Tensor,
                    device_len: torch.Tensor, table_idx: torch.Tensor, page_table: torch.Tensor,
                    max_q_len: int, sm_scale: Optional[float] = None, window: int = 0,
                    kv_begin: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_paged_attention: causal attention of the packed queries ``q`` [n, q_heads,
    head_dim] (request i's are the positions [cached_len[i], device_len[i])) over
    ``cache``.  ``max_q_len`` bounds a request's query tokens (1 for a decode step);
    ``sm_scale`` defaults to head_dim ** -0.5.  ``workspace`` (uint8, its first
    PKV_ATTENTION_ZERO_BYTES zeroed once; calls that may overlap pass different ones)
    defaults to a buffer of the stream's own (some 60 MB, kept), in a capture to one of
    the capture's.  Returns ``out`` (allocated here if not given); ``lse`` [n, q_heads]
    fp32 receives the log-sum-exp if given.  See include/pkv.h."""
    if out is None:
        out = _new_like(q, stream)
    call = (_binding or _bind()).paged_attention
    rc = call(cache._ref, cache._index, q, out, lse, cached_len, device_len, table_idx, kv_begin,
              max_q_len, page_table, sm_scale, window, status, workspace, stream,
              _attention_workspaces if workspace is None else None)
    if rc:
        if rc.__class__ is tuple:  # the stream has no workspace yet
            workspace = _default_attention_workspace(*rc, cache._index)
            rc = call(cache._ref, cache._index, q, out, lse, cached_len, device_len, table_idx,
                      kv_begin, max_q_len, page_table, sm_scale, window, status, workspace, stream,
                      None)
        _check(rc)
    return out


def adjust_logits(logits: torch.Tensor, out: Optional[torch.Tensor] = None,
                  token_pool: Optional[torch.Tensor] = None,
                  table_idx: Optional[torch.Tensor] = None,
                  prompt_len: Optional[torch.Tensor] = None,
                  device_len: Optional[torch.Tensor] = None,
                  repetition: Optional[torch.Tensor] = None,
                  presence: Optional[torch.Tensor] = None,
                  frequency: Optional[torch.Tensor] = None,
                  bias_ptr: Optional[torch.Tensor] = None,
                  bias_ids: Optional[torch.Tensor] = None,
                  bias_values: Optional[torch.Tensor] = None,
                  mask: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """pkv_adjust_logits: repetition, presence and frequency penalties over each row's
    history in ``token_pool``, then sparse biases, then a grammar bit mask
    ([B, ceil(V / 32)] int32), into ``out`` (None: in place).  Returns it.  See
    include/pkv.h."""
    if out is None:
        out = logits
    rc = (_binding or _bind()).adjust_logits(
        logits, out, token_pool, table_idx, prompt_len, device_len, repetition, presence, frequency,
        bias_ptr, bias_ids, bias_values, mask, status, stream)
    if rc:
        _check(rc)
    return out
