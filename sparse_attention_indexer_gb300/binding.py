"""Thin Python binding of the C ABI in include/topk_paged.h.

Argument marshalling only: every step of the computation runs in the CUDA library.
Functions keep the C names and argument order; pointer arguments accept CUDA torch
tensors (their data_ptr is passed) or plain integers, and `stream` accepts a
torch.cuda.Stream, a raw handle or None (the current torch stream). If the library
is missing this module raises; there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("TOPK_PAGED_LIB") or os.path.join(_PKG, "libtopk_paged.so")

TOPK_MAX_K = 2048
STATUS_LEN = 1
STATUS_TABLE_WIDTH = 2
STATUS_TABLE_ENTRY = 4
STATUS_SLOT_OVERFLOW = 8
STATUS_TIMEOUT = 16
STATUS_PLAN_MISMATCH = 32
STATUS_ORDER = 64
ERR_STATIC_ROWS = -12
STATIC_MAX_ROWS = 64

EXPORTS = (
    "topk_workspace_bytes", "topk_max_row_len", "topk_chunk_capacity", "topk_plan",
    "topk_plan_ex", "topk_select_paged", "topk_read_status", "topk_clear_status",
    "topk_status_str", "topk_grid_size", "topk_plan_host", "topk_layout_info",
    "topk_select_paged_noalloc", "indexer_k_prologue", "hisparse_resolve",
    "topk_select_paged_test", "indexer_mqa_logits", "hisparse_resolve_mtp",
    "kv8_store", "kv8_attention", "kv8_attention_selected", "kv8_attention_workspace_bytes",
    "kvpages_workspace_bytes", "kvpages_reserve", "kvpages_fork", "kvpages_free",
    "kvpages_compact", "kvpages_copy", "draft_verify",
)


class TopKError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {code} ({status_str(code)})")
        self.code = code


_lib = None

_c = ctypes
_VP = _c.c_void_p
_SIGS = {
    "topk_workspace_bytes": (_c.c_size_t, [_c.c_int, _c.c_int]),
    "topk_max_row_len": (_c.c_int64, []),
    "topk_chunk_capacity": (_c.c_int, []),
    "topk_grid_size": (_c.c_int, []),
    "topk_plan": (_c.c_int, [_VP, _c.c_int, _c.c_int, _VP, _c.c_size_t, _VP]),
    "topk_plan_ex": (_c.c_int, [_VP, _c.c_int, _c.c_int, _c.c_int, _VP, _c.c_size_t, _VP]),
    "topk_select_paged": (_c.c_int, [_VP, _c.c_int64, _VP, _c.c_int, _c.c_int, _c.c_int, _VP,
                                     _c.c_int64, _VP, _c.c_int, _VP, _VP, _VP, _VP]),
    "topk_read_status": (_c.c_int, [_VP, _VP, _c.POINTER(_c.c_int)]),
    "topk_clear_status": (_c.c_int, [_VP, _VP]),
    "topk_status_str": (_c.c_char_p, [_c.c_int]),
    "topk_plan_host": (_c.c_int, [_VP, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _VP, _c.c_size_t]),
    "topk_layout_info": (_c.c_int, [_c.c_int, _c.POINTER(_c.c_int64), _c.c_int]),
    "topk_select_paged_test": (_c.c_int, [_VP, _c.c_int64, _VP, _c.c_int, _c.c_int, _c.c_int,
                                          _VP, _c.c_int64, _VP, _c.c_int, _VP, _VP, _VP, _VP,
                                          _c.c_uint64, _c.c_int]),
    "topk_select_paged_noalloc": (_c.c_int, [_VP, _c.c_int64, _VP, _c.c_int, _c.c_int, _c.c_int,
                                             _VP, _c.c_int64, _VP, _c.c_int, _VP, _VP, _VP, _VP]),
    "indexer_k_prologue": (_c.c_int, [_VP, _c.c_int64, _c.c_int, _c.c_int, _VP, _VP, _c.c_float,
                                      _VP, _VP, _c.c_int, _c.c_int, _VP, _VP, _c.c_int,
                                      _c.c_int64, _c.c_int, _VP, _VP, _c.c_int64, _VP, _VP]),
    "indexer_mqa_logits": (_c.c_int, [_VP, _VP, _c.c_int, _c.c_int, _c.c_int, _VP, _c.c_int,
                                      _c.c_int, _VP, _VP, _c.c_int, _c.c_int, _c.c_int, _VP, _VP,
                                      _c.c_int64, _VP, _c.c_int64, _VP, _VP]),
    "hisparse_resolve": (_c.c_int, [_VP, _c.c_int, _c.c_int, _VP, _c.c_int64, _c.c_int, _VP,
                                    _c.c_int64, _VP, _VP, _VP, _c.c_int, _c.c_int, _VP, _VP,
                                    _c.c_int64, _VP, _c.c_int64, _c.c_int, _VP, _VP, _VP, _VP]),
    "hisparse_resolve_mtp": (_c.c_int, [_VP, _c.c_int, _c.c_int, _c.c_int, _VP, _c.c_int64,
                                        _c.c_int, _VP, _c.c_int64, _VP, _VP, _VP, _c.c_int,
                                        _c.c_int, _VP, _VP, _c.c_int64, _VP, _c.c_int64, _c.c_int,
                                        _VP, _VP, _VP, _VP]),
    "kv8_store": (_c.c_int, [_VP, _c.c_int64, _VP, _c.c_int64, _c.c_int, _c.c_int, _c.c_int,
                             _c.c_int, _VP, _VP, _VP, _c.c_int, _c.c_int64, _c.c_int, _c.c_int,
                             _VP, _VP, _VP, _VP, _c.c_int64, _VP, _VP]),
    "kv8_attention_workspace_bytes": (_c.c_int64, [_c.c_int, _c.c_int, _c.c_int, _c.c_int]),
    "kv8_attention": (_c.c_int, [_VP, _c.c_int64, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                                 _c.c_int, _c.c_float, _VP, _c.c_int, _c.c_int, _VP, _VP,
                                 _c.c_int, _c.c_int64, _c.c_int, _c.c_int, _VP, _VP, _VP, _VP,
                                 _c.c_int64, _VP, _c.c_int64, _VP, _VP, _c.c_int64, _VP, _VP]),
    "kv8_attention_selected": (_c.c_int, [_VP, _c.c_int64, _c.c_int, _c.c_int, _c.c_int,
                                          _c.c_int, _c.c_int, _c.c_float, _VP, _c.c_int,
                                          _c.c_int64, _c.c_int, _VP, _VP, _VP, _VP, _c.c_int64,
                                          _VP, _c.c_int64, _VP, _VP, _c.c_int64, _VP, _VP]),
    "kvpages_workspace_bytes": (_c.c_size_t, [_c.c_int, _c.c_int]),
    "kvpages_reserve": (_c.c_int, [_VP, _VP, _VP, _c.c_int, _VP, _c.c_int, _c.c_int64, _c.c_int,
                                   _VP, _c.c_int, _VP, _c.c_int, _VP, _c.c_size_t, _VP, _VP]),
    "kvpages_fork": (_c.c_int, [_VP, _VP, _VP, _c.c_int, _VP, _c.c_int, _c.c_int64, _c.c_int,
                                _VP, _c.c_int, _VP, _VP]),
    "kvpages_free": (_c.c_int, [_VP, _VP, _c.c_int, _VP, _c.c_int, _c.c_int64, _c.c_int, _VP,
                                _c.c_int, _VP, _VP]),
    "kvpages_compact": (_c.c_int, [_VP, _c.c_int, _c.c_int64, _VP, _c.c_int, _VP, _c.c_int, _VP,
                                   _VP, _VP, _c.c_size_t, _VP, _VP]),
    "kvpages_copy": (_c.c_int, [_VP, _VP, _c.c_int, _c.c_int, _VP, _c.c_int, _VP, _VP]),
    "draft_verify": (_c.c_int, [_VP, _c.c_int64, _c.c_int64, _VP, _c.c_int64, _c.c_int64, _VP,
                                _VP, _VP, _c.c_int, _c.c_int, _c.c_int, _VP, _VP, _VP, _VP]),
}

# include/hisparse_resolver.h
RESOLVER_STATUS_NO_VICTIM = 1
RESOLVER_STATUS_POSITION = 2
RESOLVER_STATUS_HOST_ROW = 4
RESOLVER_STATUS_KV_ROW = 8

# include/indexer_prologue.h
PROLOGUE_OK = 0
PROLOGUE_ERR_NULL = -1
PROLOGUE_ERR_SHAPE = -2
PROLOGUE_ERR_ALIGN = -3
PROLOGUE_ERR_CUDA = -4
PROLOGUE_STATUS_POSITION = 1
PROLOGUE_STATUS_TABLE_WIDTH = 2
PROLOGUE_STATUS_TABLE_ENTRY = 4
PROLOGUE_STATUS_SLOT = 8
PROLOGUE_STATUS_TABLE_ROW = 16


class PrologueError(RuntimeError):
    def __init__(self, code: int):
        super().__init__(f"indexer_k_prologue: {code}")
        self.code = code


def lib():
    """Loads libtopk_paged.so (built by sparse_attention_indexer_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if x.numel() > 0 and not x.is_cuda:
            raise ValueError("device pointer argument must be a CUDA tensor")
        return x.data_ptr() or None
    return int(x)


def _stream(s) -> Optional[int]:
    if s is None:
        if torch.cuda.is_initialized():  # the current stream without a Stream object
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) or None
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(s, torch.cuda.Stream):
        return s.cuda_stream or None
    return int(s) or None


def _check(code: int, what: str) -> int:
    if code < 0:
        raise TopKError(code, what)
    return code


def status_str(code: int) -> str:
    return lib().topk_status_str(int(code)).decode()


topk_status_str = status_str


def topk_workspace_bytes(rows: int, max_len: int) -> int:
    return int(lib().topk_workspace_bytes(int(rows), int(max_len)))


def topk_max_row_len() -> int:
    return int(_check(lib().topk_max_row_len(), "topk_max_row_len"))


def topk_chunk_capacity() -> int:
    return int(lib().topk_chunk_capacity())


def topk_grid_size() -> int:
    return int(_check(lib().topk_grid_size(), "topk_grid_size"))


def topk_plan(lens, rows: int, max_len: int, workspace, ws_bytes: int, stream=None) -> int:
    return _check(lib().topk_plan(_ptr(lens), int(rows), int(max_len), _ptr(workspace),
                                  int(ws_bytes), _stream(stream)), "topk_plan")


def topk_plan_ex(lens, rows: int, max_len: int, chunk: int, workspace, ws_bytes: int,
                 stream=None) -> int:
    return _check(lib().topk_plan_ex(_ptr(lens), int(rows), int(max_len), int(chunk),
                                     _ptr(workspace), int(ws_bytes), _stream(stream)),
                  "topk_plan_ex")


def topk_select_paged_test(scores, ld: int, lens, rows: int, max_len: int, k: int, block_table,
                           table_ld: int, row_to_table, page_size: int, out_slots, out_pos,
                           workspace, wait_ns: int, skip_cta: int, stream=None) -> int:
    """topk_select_paged with a bounded-wait limit (ns) and a CTA that skips the first
    row-barrier arrival of its units (test hooks)."""
    return _check(lib().topk_select_paged_test(
        _ptr(scores), int(ld), _ptr(lens), int(rows), int(max_len), int(k), _ptr(block_table),
        int(table_ld), _ptr(row_to_table), int(page_size), _ptr(out_slots), _ptr(out_pos),
        _ptr(workspace), _stream(stream), int(wait_ns), int(skip_cta)), "topk_select_paged_test")


def topk_select_paged(scores, ld: int, lens, rows: int, max_len: int, k: int, block_table,
                      table_ld: int, row_to_table, page_size: int, out_slots, out_pos,
                      workspace, stream=None) -> int:
    return _check(lib().topk_select_paged(
        _ptr(scores), int(ld), _ptr(lens), int(rows), int(max_len), int(k), _ptr(block_table),
        int(table_ld), _ptr(row_to_table), int(page_size), _ptr(out_slots), _ptr(out_pos),
        _ptr(workspace), _stream(stream)), "topk_select_paged")


def topk_select_paged_noalloc(scores, ld: int, lens, rows: int, max_len: int, k: int,
                              block_table, table_ld: int, row_to_table, page_size: int,
                              out_slots, out_pos, status, stream=None) -> int:
    """No workspace argument: the library's static device scratch serves the call."""
    return _check(lib().topk_select_paged_noalloc(
        _ptr(scores), int(ld), _ptr(lens), int(rows), int(max_len), int(k), _ptr(block_table),
        int(table_ld), _ptr(row_to_table), int(page_size), _ptr(out_slots), _ptr(out_pos),
        _ptr(status), _stream(stream)), "topk_select_paged_noalloc")


def topk_read_status(workspace, stream=None) -> int:
    v = ctypes.c_int(0)
    _check(lib().topk_read_status(_ptr(workspace), _stream(stream), ctypes.byref(v)),
           "topk_read_status")
    return int(v.value)


def topk_clear_status(workspace, stream=None) -> int:
    return _check(lib().topk_clear_status(_ptr(workspace), _stream(stream)), "topk_clear_status")


def topk_plan_host(lens, rows: int, max_len: int, grid: int, chunk: int, image) -> int:
    """Host reference of the planner writing into a host buffer (numpy uint8 array)."""
    import numpy as np
    lens = np.ascontiguousarray(lens, dtype=np.int32)
    return _check(lib().topk_plan_host(lens.ctypes.data_as(ctypes.c_void_p), int(rows),
                                       int(max_len), int(grid), int(chunk),
                                       image.ctypes.data_as(ctypes.c_void_p), int(image.nbytes)),
                  "topk_plan_host")


def indexer_k_prologue(k, ln_w, ln_b, eps: float, positions, cos_sin, rope_dim: int,
                       token_table, block_table, page_size: int, cache, cache_scale,
                       status=None, stream=None) -> int:
    """indexer_k_prologue of include/indexer_prologue.h on CUDA tensors: k (bf16 or
    its int16 bits) [tokens, ld], ln_w / ln_b float32 [dim], positions / token_table
    int32 [tokens], cos_sin float32 [max_pos, rope_dim], block_table int32
    [n_tables, table_ld], cache uint8 [num_slots, dim], cache_scale float32
    [num_slots], status int32 [1] or None. Argument marshalling only."""
    tokens, ld = (int(k.shape[0]), int(k.stride(0))) if k.dim() == 2 else (0, 0)
    dim = int(k.shape[1]) if k.dim() == 2 else 0
    code = lib().indexer_k_prologue(
        _ptr(k), ld, tokens, dim, _ptr(ln_w), _ptr(ln_b), float(eps), _ptr(positions),
        _ptr(cos_sin), int(cos_sin.shape[0]), int(rope_dim), _ptr(token_table),
        _ptr(block_table), int(block_table.shape[0]), int(block_table.stride(0)), int(page_size),
        _ptr(cache), _ptr(cache_scale), int(cache.shape[0]), _ptr(status), _stream(stream))
    if code < 0:
        raise PrologueError(code)
    return code


# include/indexer_logits.h
LOGITS_ERR_NULL = -1
LOGITS_ERR_SHAPE = -2
LOGITS_ERR_ALIGN = -3
LOGITS_ERR_CUDA = -4
LOGITS_STATUS_LEN = 1
LOGITS_STATUS_TABLE_WIDTH = 2
LOGITS_STATUS_TABLE_ENTRY = 4
LOGITS_STATUS_SLOT = 8
LOGITS_STATUS_TABLE_ROW = 16
LOGITS_STATUS_TIMEOUT = 32


class LogitsError(RuntimeError):
    def __init__(self, code: int):
        super().__init__(f"indexer_mqa_logits: {code}")
        self.code = code


def indexer_mqa_logits(q, w, lens, max_len: int, group_rows: int, group_table, block_table,
                       page_size: int, cache, cache_scale, scores, status=None,
                       stream=None) -> int:
    """indexer_mqa_logits of include/indexer_logits.h on CUDA tensors: q uint8 [rows,
    heads, dim], w float32 [rows, heads], lens int32 [rows], group_table int32 [groups]
    or None, block_table int32 [n_tables, table_ld], cache uint8 [num_slots, dim],
    cache_scale float32 [num_slots], scores float32 [rows, ld], status int32 [1] or
    None. Argument marshalling only."""
    rows, heads, dim = (int(x) for x in q.shape)
    code = lib().indexer_mqa_logits(
        _ptr(q), _ptr(w), rows, heads, dim, _ptr(lens), int(max_len), int(group_rows),
        _ptr(group_table), _ptr(block_table), int(block_table.shape[0]),
        int(block_table.stride(0)), int(page_size), _ptr(cache), _ptr(cache_scale),
        int(cache.shape[0]), _ptr(scores), int(scores.stride(0)), _ptr(status), _stream(stream))
    if code < 0:
        raise LogitsError(code)
    return code


class ResolverError(RuntimeError):
    def __init__(self, code: int):
        super().__init__(f"hisparse_resolve: {code}")
        self.code = code


def hisparse_resolve(positions, block_table, page_size: int, token_to_hot, hot_token,
                     hot_step, hot_rows, step: int, host_kv, host_base, kv, out_rows,
                     counts=None, status=None, stream=None) -> int:
    """hisparse_resolve of include/hisparse_resolver.h: positions / block_table /
    token_to_hot / hot_token / hot_step / hot_rows / out_rows CUDA int32 tensors, host_kv
    a pinned CPU uint8 tensor [host_rows, row_bytes], host_base CUDA int64 [rows], kv
    CUDA uint8 [kv_rows, row_bytes]. Argument marshalling only."""
    if host_kv.is_cuda or (host_kv.numel() and not host_kv.is_pinned()):
        raise ValueError("host_kv must be pinned host memory")
    rows, k = int(positions.shape[0]), int(positions.shape[1])
    code = lib().hisparse_resolve(
        _ptr(positions), rows, k, _ptr(block_table), int(block_table.stride(0)),
        int(page_size), _ptr(token_to_hot), int(token_to_hot.stride(0)), _ptr(hot_token),
        _ptr(hot_step), _ptr(hot_rows), int(hot_rows.shape[1]), int(step),
        host_kv.data_ptr() or None, _ptr(host_base), int(host_kv.shape[0]), _ptr(kv),
        int(kv.shape[0]), int(kv.shape[1]), _ptr(out_rows), _ptr(counts), _ptr(status),
        _stream(stream))
    if code < 0:
        raise ResolverError(code)
    return code


def hisparse_resolve_mtp(positions, block_table, page_size: int, token_to_hot, hot_token,
                         hot_step, hot_rows, step: int, host_kv, host_base, kv, out_rows,
                         counts=None, status=None, stream=None) -> int:
    """hisparse_resolve_mtp of include/hisparse_resolver.h: as hisparse_resolve, with
    positions and out_rows CUDA int32 [rows, q_rows, k]. Argument marshalling only."""
    if host_kv.is_cuda or (host_kv.numel() and not host_kv.is_pinned()):
        raise ValueError("host_kv must be pinned host memory")
    rows, q_rows, k = (int(x) for x in positions.shape)
    code = lib().hisparse_resolve_mtp(
        _ptr(positions), rows, q_rows, k, _ptr(block_table), int(block_table.stride(0)),
        int(page_size), _ptr(token_to_hot), int(token_to_hot.stride(0)), _ptr(hot_token),
        _ptr(hot_step), _ptr(hot_rows), int(hot_rows.shape[1]), int(step),
        host_kv.data_ptr() or None, _ptr(host_base), int(host_kv.shape[0]), _ptr(kv),
        int(kv.shape[0]), int(kv.shape[1]), _ptr(out_rows), _ptr(counts), _ptr(status),
        _stream(stream))
    if code < 0:
        raise ResolverError(code)
    return code


# include/kv8_attention.h
KV8_BF16 = 0
KV8_FP16 = 1
KV8_ERR_NULL = -1
KV8_ERR_SHAPE = -2
KV8_ERR_ALIGN = -3
KV8_ERR_CUDA = -4
KV8_ERR_WORKSPACE = -5
KV8_STATUS_LEN = 1
KV8_STATUS_TABLE_WIDTH = 2
KV8_STATUS_TABLE_ENTRY = 4
KV8_STATUS_SLOT = 8
KV8_STATUS_TABLE_ROW = 16
KV8_STATUS_POSITION = 32

_KV8_TYPES = {torch.bfloat16: KV8_BF16, torch.float16: KV8_FP16}


class Kv8Error(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {code}")
        self.code = code


def _kv8(code: int, what: str) -> int:
    if code < 0:
        raise Kv8Error(code, what)
    return code


def _ld(t) -> int:
    """Stride of the first dimension; a lone row's may be anything, so its length."""
    return t.stride(0) if t.shape[0] > 1 else math.prod(t.shape[1:])


def kv8_store(k, v, positions, token_table, block_table, page_size: int, block_tokens: int,
              k_cache, v_cache, k_scale, v_scale, status=None, stream=None) -> int:
    """kv8_store of include/kv8_attention.h on CUDA tensors: k, v bf16 / fp16 [tokens,
    kv_heads, dim] (rows may be strided), positions / token_table int32 [tokens],
    block_table int32 [n_tables, table_ld], caches uint8 [num_slots, kv_heads, dim],
    scales float32 [num_slots / block_tokens, kv_heads], status int32 [1] or None.
    Argument marshalling only."""
    tokens, heads, dim = k.shape
    return _kv8(lib().kv8_store(
        _ptr(k), _ld(k), _ptr(v), _ld(v), _KV8_TYPES[k.dtype], tokens, heads, dim,
        _ptr(positions), _ptr(token_table), _ptr(block_table), block_table.shape[0],
        block_table.shape[1], page_size, block_tokens, _ptr(k_cache), _ptr(v_cache),
        _ptr(k_scale), _ptr(v_scale), k_cache.shape[0], _ptr(status), _stream(stream)),
        "kv8_store")


def kv8_attention_workspace_bytes(q_heads: int, kv_heads: int, dim: int,
                                  group_rows: int) -> int:
    return _kv8(lib().kv8_attention_workspace_bytes(int(q_heads), int(kv_heads), int(dim),
                                                    int(group_rows)),
                "kv8_attention_workspace_bytes")


def kv8_attention(q, sm_scale: float, lens, max_len: int, group_rows: int, group_table,
                  block_table, page_size: int, block_tokens: int, k_cache, v_cache, k_scale,
                  v_scale, out, lse, workspace, status=None, stream=None) -> int:
    """kv8_attention of include/kv8_attention.h on CUDA tensors: q and out bf16 / fp16
    [rows, q_heads, dim] (rows may be strided), lens int32 [rows], group_table int32
    [groups] or None, lse float32 [rows, q_heads] or None, the cache as in kv8_store.
    Argument marshalling only."""
    rows, heads, dim = q.shape
    return _kv8(lib().kv8_attention(
        _ptr(q), _ld(q), _KV8_TYPES[q.dtype], rows, heads, k_cache.shape[1], dim, sm_scale,
        _ptr(lens), max_len, group_rows, _ptr(group_table), _ptr(block_table),
        block_table.shape[0], block_table.shape[1], page_size, block_tokens, _ptr(k_cache),
        _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), k_cache.shape[0], _ptr(out), _ld(out),
        _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)), "kv8_attention")


def kv8_attention_selected(q, sm_scale: float, slots, block_tokens: int, k_cache, v_cache,
                           k_scale, v_scale, out, lse, workspace, status=None,
                           stream=None) -> int:
    """kv8_attention_selected of include/kv8_attention.h: slots int32 [rows, k], the rest
    as in kv8_attention. Argument marshalling only."""
    rows, heads, dim = q.shape
    return _kv8(lib().kv8_attention_selected(
        _ptr(q), _ld(q), _KV8_TYPES[q.dtype], rows, heads, k_cache.shape[1], dim, sm_scale,
        _ptr(slots), slots.shape[1], _ld(slots), block_tokens, _ptr(k_cache),
        _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), k_cache.shape[0], _ptr(out), _ld(out),
        _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)), "kv8_attention_selected")


# include/kv_pages.h
KVPAGES_MAX_PLANES = 240
KVPAGES_ERR_NULL = -1
KVPAGES_ERR_SHAPE = -2
KVPAGES_ERR_ALIGN = -3
KVPAGES_ERR_CUDA = -4
KVPAGES_ERR_WORKSPACE = -5
KVPAGES_STATUS_ROW = 1
KVPAGES_STATUS_LEN = 2
KVPAGES_STATUS_PAGE = 4
KVPAGES_STATUS_NO_PAGE = 8
KVPAGES_STATUS_CHILD = 16
KVPAGES_STATUS_REFS = 32


class KvPlane(_c.Structure):
    """kvpages_plane of include/kv_pages.h."""
    _fields_ = [("base", _c.c_void_p), ("page_bytes", _c.c_int64)]


class KvPagesError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {code}")
        self.code = code


def _kvp(code: int, what: str) -> int:
    if code < 0:
        raise KvPagesError(code, what)
    return code


def kvpages_workspace_bytes(n: int, num_pages: int) -> int:
    return int(lib().kvpages_workspace_bytes(int(n), int(num_pages)))


def kvpages_planes(tensors, num_pages: int):
    """The plane array of the pages' tensors: CUDA tensors whose first dimension is a
    page (num_pages of them) and whose rest is contiguous."""
    planes = (KvPlane * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        if not t.is_cuda or t.shape[0] != num_pages or not t.is_contiguous():
            raise ValueError("a plane is a contiguous CUDA tensor [num_pages, ...]")
        planes[i].base = t.data_ptr()
        planes[i].page_bytes = t[0].numel() * t.element_size() if num_pages else 4
    return planes


def kvpages_reserve(rows, old_lens, new_lens, block_table, page_size: int, refs, planes,
                    n_planes: int, workspace, status=None, stream=None) -> int:
    """kvpages_reserve of include/kv_pages.h: rows / old_lens / new_lens int32 [n],
    block_table int32 [n_tables, table_ld] (contiguous), refs int32 [num_pages], planes
    from kvpages_planes. Argument marshalling only."""
    return _kvp(lib().kvpages_reserve(
        _ptr(rows), _ptr(old_lens), _ptr(new_lens), rows.shape[0], _ptr(block_table),
        block_table.shape[0], block_table.shape[1], page_size, _ptr(refs), refs.shape[0], planes,
        n_planes, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)), "kvpages_reserve")


def kvpages_fork(parents, children, lens, block_table, page_size: int, refs, status=None,
                 stream=None) -> int:
    """kvpages_fork of include/kv_pages.h (arguments as in kvpages_reserve)."""
    return _kvp(lib().kvpages_fork(
        _ptr(parents), _ptr(children), _ptr(lens), parents.shape[0], _ptr(block_table),
        block_table.shape[0], block_table.shape[1], page_size, _ptr(refs), refs.shape[0],
        _ptr(status), _stream(stream)), "kvpages_fork")


def kvpages_free(rows, keep_lens, block_table, page_size: int, refs, status=None,
                 stream=None) -> int:
    """kvpages_free of include/kv_pages.h: keep_lens int32 [n] or None (keeps nothing)."""
    return _kvp(lib().kvpages_free(
        _ptr(rows), _ptr(keep_lens), rows.shape[0], _ptr(block_table), block_table.shape[0],
        block_table.shape[1], page_size, _ptr(refs), refs.shape[0], _ptr(status),
        _stream(stream)), "kvpages_free")


def kvpages_compact(block_table, refs, planes, n_planes: int, new_ids, counts, workspace,
                    status=None, stream=None) -> int:
    """kvpages_compact of include/kv_pages.h: new_ids int32 [num_pages], counts int32 [2]
    or None."""
    return _kvp(lib().kvpages_compact(
        _ptr(block_table), block_table.shape[0], block_table.shape[1], _ptr(refs),
        refs.shape[0], planes, n_planes, _ptr(new_ids), _ptr(counts), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)),
        "kvpages_compact")


def kvpages_copy(src, dst, num_pages: int, planes, n_planes: int, status=None,
                 stream=None) -> int:
    """kvpages_copy of include/kv_pages.h: src / dst int32 [n]."""
    return _kvp(lib().kvpages_copy(_ptr(src), _ptr(dst), src.shape[0], num_pages, planes,
                                   n_planes, _ptr(status), _stream(stream)), "kvpages_copy")


# include/draft_verify.h
VERIFY_MAX_DRAFTS = 31
VERIFY_ERR_NULL = -1
VERIFY_ERR_SHAPE = -2
VERIFY_ERR_ALIGN = -3
VERIFY_ERR_CUDA = -4
VERIFY_STATUS_COUNT = 1
VERIFY_STATUS_TOKEN = 2
VERIFY_STATUS_PROB = 4
VERIFY_STATUS_EMPTY = 8
VERIFY_STATUS_UNIFORM = 16


class VerifyError(RuntimeError):
    def __init__(self, code: int):
        super().__init__(f"draft_verify: {code}")
        self.code = code


def draft_verify(target, draft, tokens, uniforms, out_tokens, kept, n_drafts=None, status=None,
                 stream=None) -> int:
    """draft_verify of include/draft_verify.h on CUDA tensors: target float32 [reqs,
    drafts + 1, vocab] and draft float32 [reqs, drafts, vocab] or None (last dimension
    contiguous), tokens int32 [reqs, drafts], uniforms float32 [reqs, drafts + 1],
    out_tokens int32 [reqs, drafts + 1], kept int32 [reqs], n_drafts int32 [reqs] or
    None. Argument marshalling only."""
    reqs, drafts = tokens.shape
    vocab = target.shape[2]
    # the stride of a dimension of one row may be anything
    row = lambda t: t.stride(1) if t is not None and t.shape[1] > 1 else vocab  # noqa: E731
    code = lib().draft_verify(
        _ptr(target), target.stride(0), row(target), _ptr(draft),
        draft.stride(0) if draft is not None else 0, row(draft),
        _ptr(tokens), _ptr(n_drafts), _ptr(uniforms), reqs, drafts, vocab,
        _ptr(out_tokens), _ptr(kept), _ptr(status), _stream(stream))
    if code < 0:
        raise VerifyError(code)
    return code


def topk_layout_info(rows: int):
    arr = (ctypes.c_int64 * 12)()
    _check(lib().topk_layout_info(int(rows), arr, 12), "topk_layout_info")
    keys = ("max_grid", "max_waves", "chunk_cap", "header_bytes", "rowinfo", "singles",
            "first_single", "units", "groups", "threads", "group_cap", "list_cap")
    return dict(zip(keys, [int(v) for v in arr]))
