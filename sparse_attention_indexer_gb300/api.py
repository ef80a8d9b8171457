"""Tensor-level front end over the C ABI: workspace ownership, plan reuse, host I/O.

Every compute step runs in the CUDA library (libtopk_paged.so); this module only
allocates device memory through torch and passes pointers, sizes and the stream.
"""
from __future__ import annotations

import contextlib
import threading
from typing import Optional, Sequence, Tuple

import torch

from . import binding as B


class PagedTopK:
    """Top-k selection with paged slot translation for batches of up to `rows` rows
    whose valid lengths are at most `max_len`.

    plan() is called once per batch (per forward); select() once per indexer layer,
    any k in [1, 2048]. Output rows hold min(k, len) slots then -1."""

    def __init__(self, rows: int, max_len: int, device: Optional[torch.device] = None):
        if device is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.rows = int(rows)
        self.max_len = int(max_len)
        self.device = device
        self.ws_bytes = B.topk_workspace_bytes(self.rows, self.max_len)
        # torch's caching allocator returns 512-byte aligned blocks
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        assert self.workspace.data_ptr() % 256 == 0

    def plan(self, lens: torch.Tensor, chunk: int = 0, stream=None) -> None:
        """chunk forces the elements per CTA when nonzero (tests: path forcing)."""
        assert lens.dtype == torch.int32 and lens.is_cuda and lens.numel() == self.rows
        if chunk:
            B.topk_plan_ex(lens, self.rows, self.max_len, chunk, self.workspace, self.ws_bytes,
                           stream)
        else:
            B.topk_plan(lens, self.rows, self.max_len, self.workspace, self.ws_bytes, stream)

    def select(self, scores: torch.Tensor, lens: torch.Tensor, k: int, block_table: torch.Tensor,
               page_size: int, row_to_table: Optional[torch.Tensor] = None,
               out_slots: Optional[torch.Tensor] = None, out_pos: Optional[torch.Tensor] = None,
               with_pos: bool = False, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        assert scores.dtype == torch.float32 and scores.dim() == 2 and scores.stride(1) == 1
        assert scores.shape[0] == self.rows
        assert block_table.dtype == torch.int32 and block_table.dim() == 2
        assert block_table.stride(1) == 1
        if out_slots is None:
            out_slots = torch.empty((self.rows, k), dtype=torch.int32, device=scores.device)
        if with_pos and out_pos is None:
            out_pos = torch.empty((self.rows, k), dtype=torch.int32, device=scores.device)
        B.topk_select_paged(scores, scores.stride(0), lens, self.rows, self.max_len, k,
                            block_table, block_table.stride(0), row_to_table, page_size,
                            out_slots, out_pos, self.workspace, stream)
        return out_slots, out_pos

    def status(self, stream=None) -> int:
        return B.topk_read_status(self.workspace, stream)

    def clear_status(self, stream=None) -> None:
        B.topk_clear_status(self.workspace, stream)


class HostPagedTopK:
    """End-to-end call on host buffers: pinned host -> device copies, plan + select,
    device -> pinned host copy of the slots, all on one stream."""

    def __init__(self, rows: int, ld: int, max_len: int, k: int, n_tables: int, table_ld: int,
                 with_row_to_table: bool, device: Optional[torch.device] = None):
        self.core = PagedTopK(rows, max_len, device)
        dev = self.core.device
        self.k = int(k)
        self.scores = torch.empty((rows, ld), dtype=torch.float32, device=dev)
        self.lens = torch.empty(rows, dtype=torch.int32, device=dev)
        self.table = torch.empty((n_tables, table_ld), dtype=torch.int32, device=dev)
        self.r2t = (torch.empty(rows, dtype=torch.int32, device=dev) if with_row_to_table
                    else None)
        self.out = torch.empty((rows, k), dtype=torch.int32, device=dev)
        self.out_host = torch.empty((rows, k), dtype=torch.int32, pin_memory=True)

    def h2d_bytes(self, with_table: bool = True) -> int:
        b = self.scores.numel() * 4 + self.lens.numel() * 4
        if with_table:
            b += self.table.numel() * 4 + (self.r2t.numel() * 4 if self.r2t is not None else 0)
        return b

    def d2h_bytes(self) -> int:
        return self.out.numel() * 4

    def __call__(self, scores_h: torch.Tensor, lens_h: torch.Tensor, table_h: torch.Tensor,
                 r2t_h: Optional[torch.Tensor], page_size: int, copy_table: bool = True,
                 stream=None) -> torch.Tensor:
        self.scores.copy_(scores_h, non_blocking=True)
        self.lens.copy_(lens_h, non_blocking=True)
        if copy_table:
            self.table.copy_(table_h, non_blocking=True)
            if self.r2t is not None:
                self.r2t.copy_(r2t_h, non_blocking=True)
        self.core.plan(self.lens, stream=stream)
        self.core.select(self.scores, self.lens, self.k, self.table, page_size, self.r2t,
                         out_slots=self.out, stream=stream)
        self.out_host.copy_(self.out, non_blocking=True)
        return self.out_host


class _Handle:
    """The buffers that a handle makes for itself, and the device and streams that it serves."""

    def _own(self, device: int, *tensors: torch.Tensor) -> None:
        self._device, self._buffers, self._streams = device, tensors, {B._stream(None)}

    def _stream(self, stream) -> Optional[int]:
        """The raw stream of a call. The buffers come from the pool of the stream they were made
        on, which must not give them out again while another one still works on them."""
        device = _current_device()
        if device != self._device:  # the library launches on the current device
            raise ValueError(f"the current device is not the handle's, {self._device}")
        handle = B._stream(stream) if stream is not None else _raw_stream(device) or None
        if handle not in self._streams:
            for t in self._buffers:
                t.record_stream(_torch_stream(stream))
            self._streams.add(handle)
        return handle


class Kv8Cache(_Handle):
    """A paged K/V cache in 8 bits and the attention over it (include/kv8_attention.h).

    k, v      uint8 [num_slots, kv_heads, dim]: e4m3 codes
    k_scale, v_scale  float32 [num_slots / block_tokens, kv_heads]
    The tensors stay the caller's; several layers are several caches. The workspace is made
    when a call first needs it, one for each stream the cache is used on. A call captured by
    torch.cuda.graph takes it from the graph's pool, so that graphs may be replayed on any
    streams (a capture made by other means has no such pool: use the binding there, with a
    workspace for each graph). Several host threads may call one cache, on one stream too.
    `status` collects the device status bits of all calls."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, page_size: int, block_tokens: int):
        for c, s in ((k, k_scale), (v, v_scale)):
            if c.dtype != torch.uint8 or c.dim() != 3 or not c.is_cuda or not c.is_contiguous():
                raise ValueError("a cache is a contiguous CUDA uint8 tensor [slots, heads, dim]")
            if block_tokens < 1 or c.shape[0] % block_tokens:
                raise ValueError("the slots are not a whole number of blocks")
            if (s.dtype != torch.float32 or s.device != c.device or not s.is_contiguous()
                    or tuple(s.shape) != (c.shape[0] // block_tokens, c.shape[1])):
                raise ValueError("scales are contiguous float32 [slots / block_tokens, heads]")
        if k.shape != v.shape or k.device != v.device:
            raise ValueError("k and v differ in shape or device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_size, self.block_tokens = int(page_size), int(block_tokens)
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._own(k.get_device(), self.status)
        self._workspaces = {}
        # held over an attention call: its two launches use the stream's workspace together
        self._lock = threading.Lock()
        self._heads, self._dim = k.shape[1], k.shape[2]
        # the cache's part of every call, made once
        self._args = (k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                      k.shape[0])
        self._lib = B.lib()

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, dim: int,
              block_tokens: Optional[int] = None, device: Optional[torch.device] = None):
        """A cache of num_pages pages holding zeros; block_tokens defaults to the page."""
        device = device or torch.device("cuda", torch.cuda.current_device())
        block = page_size if block_tokens is None else block_tokens
        if block < 1 or page_size % block:
            raise ValueError("page_size is not a multiple of block_tokens")
        slots = num_pages * page_size
        code = lambda: torch.zeros((slots, kv_heads, dim), dtype=torch.uint8, device=device)  # noqa: E731
        scale = lambda: torch.ones((slots // block, kv_heads), device=device)  # noqa: E731
        return cls(code(), code(), scale(), scale(), page_size, block)

    def planes(self) -> list:
        """The cache's tensors page by page, for KvPages."""
        n = self.k.shape[0] // self.page_size
        return [t.view(n, -1) for t in (self.k, self.v, self.k_scale, self.v_scale)]

    def store(self, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
              token_table: torch.Tensor, block_table: torch.Tensor, stream=None) -> None:
        """Quantises k, v [tokens, kv_heads, dim] (bf16 or fp16) into the cache."""
        tokens = k.shape[0]
        if k.shape != v.shape or k.dtype != v.dtype or k.shape[1:] != self.k.shape[1:]:
            raise ValueError("k and v are [tokens, kv_heads, dim] of one type")
        _rows(k, "k", self._device)
        _rows(v, "v", self._device)
        _int32(positions, (tokens,), "positions", self._device)
        _int32(token_table, (tokens,), "token_table", self._device)
        _table(block_table, self._device)
        code = self._lib.kv8_store(
            k.data_ptr(), B._ld(k), v.data_ptr(), B._ld(v), B._KV8_TYPES[k.dtype], tokens,
            self._heads, self._dim, positions.data_ptr(), token_table.data_ptr(),
            block_table.data_ptr(), block_table.shape[0], block_table.shape[1], self.page_size,
            self.block_tokens, *self._args, self.status.data_ptr(), self._stream(stream))
        if code < 0:
            raise B.Kv8Error(code, "kv8_store")

    def attention(self, q: torch.Tensor, lens: torch.Tensor, max_len: int,
                  block_table: torch.Tensor, sm_scale: float, group_rows: int = 1,
                  group_table: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Row t of q [rows, q_heads, dim] attends to positions [0, lens[t]) of its
        group's block-table row. Returns (out, lse)."""
        _rows(q, "q", self._device)
        rows, heads, dim = q.shape
        _int32(lens, (rows,), "lens", self._device)
        _table(block_table, self._device)
        if group_table is not None:
            _int32(group_table, (-(-rows // max(1, group_rows)),), "group_table", self._device)
        handle = self._stream(stream)
        out, lse = self._outputs(q, out, lse, stream)
        with self._lock:
            ws, ws_bytes, _held = self._workspace(heads, group_rows, handle, stream)
            code = self._lib.kv8_attention(
                q.data_ptr(), B._ld(q), B._KV8_TYPES[q.dtype], rows, heads, self._heads, dim,
                sm_scale, lens.data_ptr(), max_len, group_rows,
                None if group_table is None else group_table.data_ptr(), block_table.data_ptr(),
                block_table.shape[0], block_table.shape[1], self.page_size, self.block_tokens,
                *self._args, out.data_ptr(), B._ld(out), lse.data_ptr(), ws, ws_bytes,
                self.status.data_ptr(), handle)
        if code < 0:
            raise B.Kv8Error(code, "kv8_attention")
        return out, lse

    def attention_selected(self, q: torch.Tensor, slots: torch.Tensor, sm_scale: float,
                           out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None,
                           stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Row t of q attends to the slots of slots[t] (int32 [rows, k], negative ones
        skipped): what PagedTopK.select returns. Returns (out, lse)."""
        _rows(q, "q", self._device)
        rows, heads, dim = q.shape
        if (slots.dtype != torch.int32 or slots.dim() != 2 or slots.shape[0] != rows
                or slots.get_device() != self._device or not _last_contiguous(slots)):
            raise ValueError("slots is CUDA int32 [rows, k]")
        handle = self._stream(stream)
        out, lse = self._outputs(q, out, lse, stream)
        with self._lock:
            ws, ws_bytes, _held = self._workspace(heads, 1, handle, stream)
            code = self._lib.kv8_attention_selected(
                q.data_ptr(), B._ld(q), B._KV8_TYPES[q.dtype], rows, heads, self._heads, dim,
                sm_scale, slots.data_ptr(), slots.shape[1], B._ld(slots), self.block_tokens,
                *self._args, out.data_ptr(), B._ld(out), lse.data_ptr(), ws, ws_bytes,
                self.status.data_ptr(), handle)
        if code < 0:
            raise B.Kv8Error(code, "kv8_attention_selected")
        return out, lse

    def _outputs(self, q, out, lse, stream):
        if q.shape[2] != self._dim:
            raise ValueError("q and the cache differ in dim")
        if out is None or lse is None:
            with _on(stream):
                made = (torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None else out,
                        torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
                        if lse is None else lse)
        else:
            made = (out, lse)
        if out is not None:
            if out.shape != q.shape or out.dtype != q.dtype:
                raise ValueError("out has q's shape and type")
            _rows(out, "out", self._device)
        if lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32
                                or lse.get_device() != self._device or not lse.is_contiguous()):
            raise ValueError("lse is contiguous CUDA float32 [rows, q_heads]")
        return made

    def _workspace(self, heads, group_rows, handle, stream):
        """(pointer, bytes, tensor) of a workspace for these heads: the stream's, or in a capture
        one of the graph's own, which the caller holds until the call is enqueued."""
        with _on(stream):
            if not _capturing():
                key = (handle, heads, group_rows)
                ws = self._workspaces.get(key)
                if ws is None:
                    ws = self._workspaces[key] = self._new_workspace(heads, group_rows)
                return ws
            return self._new_workspace(heads, group_rows)

    def _new_workspace(self, heads, group_rows):
        n = B.kv8_attention_workspace_bytes(heads, self._heads, self._dim, group_rows)
        t = torch.empty(n, dtype=torch.uint8, device=self.k.device)
        return t.data_ptr(), n, t


class KvPages(_Handle):
    """Ownership of the pages of one or more paged tensors (include/kv_pages.h).

    block_table  int32 [n_tables, table_ld]: -1 where a sequence has no page
    refs         int32 [num_pages]: owners of each page, 0 of a free one
    planes       the tensors that hold the pages' data, each [num_pages, ...]
    max_rows     the most rows that one reserve names
    All stay the caller's and are changed in place. One instance serves one stream at a
    time (the replays of a graph that captured its calls among them); several host threads may
    call it there. `status` collects the device status bits of all calls."""

    def __init__(self, block_table: torch.Tensor, refs: torch.Tensor, page_size: int,
                 planes: Sequence[torch.Tensor] = (), max_rows: int = 1024):
        if not block_table.is_cuda:
            raise ValueError("block_table is a CUDA tensor")
        device = block_table.get_device()
        _table(block_table, device)
        _int32(refs, (refs.numel(),), "refs", device)
        self.block_table, self.refs, self.page_size = block_table, refs, int(page_size)
        self.num_pages = refs.shape[0]
        self.tensors = list(planes)  # keeps the planes' memory alive
        if any(t.get_device() != device for t in self.tensors):
            raise ValueError("the planes lie on another device than block_table")
        self._planes = B.kvpages_planes(self.tensors, self.num_pages)
        self.max_rows = int(max_rows)
        dev = refs.device
        self.workspace = torch.empty(B.kvpages_workspace_bytes(self.max_rows, self.num_pages),
                                     dtype=torch.uint8, device=dev)
        self.new_ids = torch.empty(self.num_pages, dtype=torch.int32, device=dev)
        self.counts = torch.zeros(2, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._own(device, self.workspace, self.new_ids, self.counts, self.status)
        # the state's part of the calls, made once
        self._table_args = (block_table.data_ptr(), block_table.shape[0], block_table.shape[1])
        self._pool_args = (refs.data_ptr(), self.num_pages)
        self._plane_args = (self._planes, len(self.tensors))
        self._ws_args = (self.workspace.data_ptr(), self.workspace.numel())
        self._status = self.status.data_ptr()
        self._lib = B.lib()
        # held over a call: reserve's and compact's two launches use the workspace together
        self._lock = threading.Lock()

    def reserve(self, rows: torch.Tensor, old_lens: torch.Tensor, new_lens: torch.Tensor,
                stream=None) -> None:
        """Makes positions [old_lens[i], new_lens[i]) of rows[i] writable."""
        n = rows.shape[0]
        for t, name in ((rows, "rows"), (old_lens, "old_lens"), (new_lens, "new_lens")):
            _int32(t, (n,), name, self._device)
        if n > self.max_rows:
            raise ValueError(f"more than max_rows = {self.max_rows} rows")
        with self._lock:
            code = self._lib.kvpages_reserve(
                rows.data_ptr(), old_lens.data_ptr(), new_lens.data_ptr(), n, *self._table_args,
                self.page_size, *self._pool_args, *self._plane_args, *self._ws_args, self._status,
                self._stream(stream))
        B._kvp(code, "kvpages_reserve")

    def fork(self, parents: torch.Tensor, children: torch.Tensor, lens: torch.Tensor,
             stream=None) -> None:
        """children[i] shares the pages of the first lens[i] positions of parents[i]."""
        n = parents.shape[0]
        for t, name in ((parents, "parents"), (children, "children"), (lens, "lens")):
            _int32(t, (n,), name, self._device)
        with self._lock:
            code = self._lib.kvpages_fork(
                parents.data_ptr(), children.data_ptr(), lens.data_ptr(), n, *self._table_args,
                self.page_size, *self._pool_args, self._status, self._stream(stream))
        B._kvp(code, "kvpages_fork")

    def free(self, rows: torch.Tensor, keep_lens: Optional[torch.Tensor] = None,
             stream=None) -> None:
        """rows[i] gives up its pages past the first keep_lens[i] positions (all of them)."""
        _int32(rows, (rows.shape[0],), "rows", self._device)
        if keep_lens is not None:
            _int32(keep_lens, (rows.shape[0],), "keep_lens", self._device)
        with self._lock:
            code = self._lib.kvpages_free(
                rows.data_ptr(), None if keep_lens is None else keep_lens.data_ptr(),
                rows.shape[0], *self._table_args, self.page_size, *self._pool_args, self._status,
                self._stream(stream))
        B._kvp(code, "kvpages_free")

    def compact(self, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Moves the live pages into the lowest ids. Returns (new_ids, counts): the new id
        of each page (-1 of a free one) and {live pages, pages moved}; both are this
        instance's buffers, overwritten by the next call."""
        with self._lock:
            code = self._lib.kvpages_compact(
                *self._table_args, *self._pool_args, *self._plane_args, self.new_ids.data_ptr(),
                self.counts.data_ptr(), *self._ws_args, self._status, self._stream(stream))
        B._kvp(code, "kvpages_compact")
        return self.new_ids, self.counts

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copies page src[i] to page dst[i] in every plane."""
        n = src.shape[0]
        _int32(src, (n,), "src", self._device)
        _int32(dst, (n,), "dst", self._device)
        with self._lock:
            code = self._lib.kvpages_copy(
                src.data_ptr(), dst.data_ptr(), n, self.num_pages, *self._plane_args, self._status,
                self._stream(stream))
        B._kvp(code, "kvpages_copy")


def verify_drafts(target: torch.Tensor, draft: Optional[torch.Tensor], tokens: torch.Tensor,
                  uniforms: torch.Tensor, n_drafts: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Speculative sampling's verification (include/draft_verify.h): target float32 [reqs,
    drafts + 1, vocab], draft float32 [reqs, drafts, vocab] or None (point masses), tokens
    int32 [reqs, drafts], uniforms float32 [reqs, drafts + 1]. Returns (out_tokens [reqs,
    drafts + 1], kept [reqs]): the kept drafts, one drawn token, then -1."""
    if tokens.dim() != 2 or not tokens.is_cuda:
        raise ValueError("tokens is CUDA int32 [reqs, drafts]")
    reqs, drafts = tokens.shape
    device = tokens.get_device()
    _int32(tokens, (reqs, drafts), "tokens", device)
    if (target.dtype != torch.float32 or target.dim() != 3 or target.get_device() != device
            or target.shape[0] != reqs or target.shape[1] != drafts + 1
            or not _last_contiguous(target)):
        raise ValueError("target is CUDA float32 [reqs, drafts + 1, vocab]")
    vocab = target.shape[2]
    if draft is not None and (draft.dtype != torch.float32 or draft.shape != (reqs, drafts, vocab)
                              or draft.get_device() != device or not _last_contiguous(draft)):
        raise ValueError("draft is CUDA float32 [reqs, drafts, vocab]")
    if (uniforms.dtype != torch.float32 or uniforms.shape != (reqs, drafts + 1)
            or uniforms.get_device() != device or not uniforms.is_contiguous()):
        raise ValueError("uniforms is contiguous CUDA float32 [reqs, drafts + 1]")
    if n_drafts is not None:
        _int32(n_drafts, (reqs,), "n_drafts", device)
    if status is not None:
        _int32(status, (1,), "status", device)
    if device != _current_device():  # where the library launches
        raise ValueError(f"the current device is not the tensors', {device}")
    with _on(stream):
        out = torch.empty((reqs, drafts + 1), dtype=torch.int32, device=tokens.device)
        kept = torch.empty((reqs,), dtype=torch.int32, device=tokens.device)
    code = B.lib().draft_verify(
        target.data_ptr(), target.stride(0), target.stride(1) if drafts else vocab,
        None if draft is None else draft.data_ptr(), 0 if draft is None else draft.stride(0),
        vocab if draft is None or drafts <= 1 else draft.stride(1), tokens.data_ptr(),
        None if n_drafts is None else n_drafts.data_ptr(), uniforms.data_ptr(), reqs, drafts,
        vocab, out.data_ptr(), kept.data_ptr(), None if status is None else status.data_ptr(),
        B._stream(stream))
    if code < 0:
        raise B.VerifyError(code)
    return out, kept


_HERE = contextlib.nullcontext()
# without the calls of Python between: they are asked for at each call of an operator
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing


def _on(stream):
    """Memory for work on `stream` comes from that stream's pool."""
    return _HERE if stream is None else torch.cuda.stream(_torch_stream(stream))


def _torch_stream(stream):
    """The torch stream of a `stream` argument."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


# `device`: the index of the GPU that a handle's (or a call's other) tensors lie on
def _int32(t: torch.Tensor, shape, name: str, device: int) -> None:
    if (t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous()
            or t.get_device() != device):
        raise ValueError(f"{name} is contiguous int32 {list(shape)} on device {device}")


def _rows(t: torch.Tensor, name: str, device: int) -> None:
    """[rows, heads, dim] of bf16 / fp16 whose rows may be strided."""
    if t.dtype not in B._KV8_TYPES or t.dim() != 3 or t.get_device() != device:
        raise ValueError(f"{name} is bf16 or fp16 [rows, heads, dim] on device {device}")
    if t.numel() and (not _last_contiguous(t) or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
        raise ValueError(f"{name}: a row's heads are contiguous")


def _table(t: torch.Tensor, device: int) -> None:
    # table_ld is a row's width as well as its stride
    if (t.dtype != torch.int32 or t.dim() != 2 or not t.is_contiguous()
            or t.get_device() != device):
        raise ValueError("block_table is contiguous int32 [n_tables, table_ld] on the handle's "
                         "device")


def _last_contiguous(t: torch.Tensor) -> bool:
    return t.shape[-1] <= 1 or t.numel() == 0 or t.stride(-1) == 1
