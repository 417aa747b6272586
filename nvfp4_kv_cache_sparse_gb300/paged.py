"""Binding of the calls on sequences in pages (``include/nvfp4_mla.h``, "Sequences in pages"): attention
over whole sequences through a page table, and the operations on the pages. Argument marshalling only,
as in the package's other calls.

A batch of sequences is ``page_table`` (int32 [batch, max_pages], inner stride 1, -1 behind a sequence's
last page), ``seq_lens`` (int32 [batch]) and ``page_refs`` (int32 [num_pages], how many table entries name
each page; a page is free when its count is 0), all on the device. ``caches`` is a list of uint8
[num_pages * page_size, record bytes] tensors, one per layer. The calls work on the tensors' own device,
whichever is current, and on ``stream`` (default: that device's current stream); workspaces that a call
makes itself belong to that stream."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple

import torch

from . import D_QK, D_V, RECORD_BYTES, _check, _need, _ptr, _record_code, load


def _stream_of(dev: int, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)   # current_stream(dev).cuda_stream builds an object for it (1 us more)
    _need(stream.device_index == dev, "the stream belongs to another device than the tensors")
    return stream.cuda_stream


def _empty(shape, dtype, dev: int, stream) -> torch.Tensor:
    """A tensor whose memory belongs to the stream that the call works on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _call(name: str, dev: int, *args) -> None:
    if torch.cuda.current_device() == dev:
        _check(name, getattr(load(), name)(*args))
    else:
        with torch.cuda.device(dev):
            _check(name, getattr(load(), name)(*args))


def _workspace(workspace: Optional[torch.Tensor], need: int, dev: int, stream) -> Tuple[torch.Tensor, int]:
    """(workspace, its bytes)"""
    if workspace is None:
        return _empty(need, torch.uint8, dev, stream), need
    _need(workspace.get_device() == dev and workspace.is_contiguous(), "workspace: contiguous, on the tensors' device")
    return workspace, workspace.numel() * workspace.element_size()


def _table(page_table: torch.Tensor, seq_lens: torch.Tensor, name: str = "page_table") -> Tuple[int, int, int]:
    """(batch, max_pages, row stride)"""
    _need(page_table.dtype == torch.int32 and page_table.dim() == 2 and (page_table.shape[1] <= 1 or page_table.stride(1) == 1),
          name + " int32 [batch, max_pages], inner stride 1")
    b, w = page_table.shape
    _need(seq_lens.dtype == torch.int32 and seq_lens.dim() == 1 and seq_lens.shape[0] == b and seq_lens.is_contiguous(),
          "seq_lens int32 [batch] contiguous")
    stride = page_table.stride(0) if b > 1 else max(w, 1)
    _need(stride >= w, name + " rows overlap")
    return b, w, stride


def _refs(page_refs: torch.Tensor) -> int:
    _need(page_refs.dtype == torch.int32 and page_refs.dim() == 1 and page_refs.is_contiguous(), "page_refs int32 [num_pages] contiguous")
    return page_refs.shape[0]


def _pool(caches: Sequence[torch.Tensor], num_pages: Optional[int], page_size: int, dev: Optional[int]):
    """(host array of the caches' pointers, number, pages, record bytes, device)"""
    _need(page_size > 0, "page_size is a power of two")
    shape, ptrs = None, []
    for c in caches:
        if shape is None:
            _need(c.dtype == torch.uint8 and c.dim() == 2 and c.is_contiguous() and c.shape[1] in RECORD_BYTES,
                  "caches: uint8 [num_slots, 352|432|656] contiguous")
            shape = c.shape
            if num_pages is None:
                num_pages = shape[0] // page_size
            if dev is None:
                dev = c.get_device()
            _need(shape[0] >= num_pages * page_size, "caches hold fewer pages than page_refs counts")
        elif c.dtype != torch.uint8 or c.shape != shape or not c.is_contiguous():
            raise ValueError("caches: contiguous uint8 tensors of one shape")
        if c.get_device() != dev or dev < 0:
            raise ValueError("all tensors on the same CUDA device")
        ptrs.append(c.data_ptr())
    return (ctypes.c_void_p * len(ptrs))(*ptrs), len(ptrs), num_pages, 352 if shape is None else shape[1], dev


def _same_device(dev: int, *tensors: Optional[torch.Tensor]) -> None:
    for t in tensors:
        if t is not None and t.get_device() != dev or dev < 0:
            raise ValueError("all tensors on the same CUDA device")


def _status(dev_status: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    _need(dev_status is None or (dev_status.dtype == torch.int32 and dev_status.numel() >= 1), "dev_status int32 [1]")
    return dev_status


def _pairs(src: torch.Tensor, dst: torch.Tensor) -> int:
    for t in (src, dst):
        _need(t.dtype == torch.int32 and t.dim() == 1 and t.is_contiguous(), "src, dst int32 [n] contiguous")
    _need(src.shape == dst.shape, "src and dst differ in length")
    return src.shape[0]


@functools.lru_cache(maxsize=256)
def paged_workspace_size(batch: int, s_q: int, h_q: int) -> int:
    """Workspace bytes of paged_mla_decode."""
    n = ctypes.c_size_t(0)
    _check("nvfp4_paged_mla_decode_workspace_size", load().nvfp4_paged_mla_decode_workspace_size(batch, s_q, h_q, ctypes.byref(n)))
    return int(n.value)


@functools.lru_cache(maxsize=256)
def pages_workspace_size(batch: int, max_pages: int, num_pages: int, num_pairs: int = 0) -> int:
    """Workspace bytes that are enough for fork_sequences, resize_sequences and compact_pages of these sizes."""
    n = ctypes.c_size_t(0)
    _check("nvfp4_mla_pages_workspace_size", load().nvfp4_mla_pages_workspace_size(batch, max_pages, num_pages, num_pairs, ctypes.byref(n)))
    return int(n.value)


def paged_mla_decode(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, sm_scale: float,
                     page_size: int = 64, attn_sink: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None, block_scales: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the last s_q tokens of each sequence over its tokens up to their own position. q bf16
    [B, s_q, h_q, 576] with 1 to 128 heads, cache uint8 [num_pages * page_size, 352|432]; returns (out bf16
    [B, s_q, h_q, 512], lse fp32 [B, s_q, h_q]). A query without a visible token gets out = 0, lse = -inf.
    ``block_scales``: the cache holds 352-byte records with their scales in block order."""
    _need(q.dtype == torch.bfloat16 and q.dim() == 4 and q.shape[3] == D_QK and q.is_contiguous(), "q bf16 [B,s_q,h_q,576] contiguous")
    B, s_q, h_q, _ = q.shape
    b, width, stride = _table(page_table, seq_lens)
    _need(b == B, "q and page_table disagree about the batch")
    _need(cache.dtype == torch.uint8 and cache.dim() == 2 and cache.is_contiguous() and cache.shape[1] in (352, 432),
          "cache uint8 [num_slots, 352|432] contiguous")
    _need(page_size > 0, "page_size is a power of two")
    code = _record_code(cache, block_scales)
    if attn_sink is not None:
        _need(attn_sink.dtype == torch.float32 and attn_sink.numel() == h_q and attn_sink.is_contiguous(), "attn_sink fp32 [h_q]")
    dev = q.get_device()   # -1 for a CPU tensor
    _same_device(dev, cache, page_table, seq_lens, attn_sink, out, lse, _status(dev_status))
    if out is None:
        out = _empty((B, s_q, h_q, D_V), torch.bfloat16, dev, stream)
    else:
        _need(out.dtype == torch.bfloat16 and out.is_contiguous() and out.shape == (B, s_q, h_q, D_V), "out bf16 [B,s_q,h_q,512]")
    if lse is None:
        lse = _empty((B, s_q, h_q), torch.float32, dev, stream)
    else:
        _need(lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == (B, s_q, h_q), "lse fp32 [B,s_q,h_q]")
    ws, ws_bytes = _workspace(workspace, paged_workspace_size(B, s_q, h_q), dev, stream)
    _call("nvfp4_paged_mla_decode", dev, q.data_ptr(), cache.data_ptr(), cache.shape[0] // page_size, page_size, code,
          page_table.data_ptr(), stride, width, seq_lens.data_ptr(), B, s_q, h_q, float(sm_scale), _ptr(attn_sink),
          out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws_bytes, _ptr(dev_status), _stream_of(dev, stream))
    return out, lse


def copy_pages(caches: Sequence[torch.Tensor], src: torch.Tensor, dst: torch.Tensor, page_size: int = 64,
               dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy page ``src[k]`` to page ``dst[k]`` (int32 [n]) in every cache. Targets should be distinct and
    none of them a source; pairs with a negative page are skipped."""
    arr, num, pages, width, dev = _pool(caches, None, page_size, None)
    _need(num > 0, "caches: at least one")
    n = _pairs(src, dst)
    _same_device(dev, src, dst, _status(dev_status))
    _call("nvfp4_mla_copy_pages", dev, arr, num, pages, page_size, width, src.data_ptr(), dst.data_ptr(), n,
          _ptr(dev_status), _stream_of(dev, stream))


def fork_sequences(page_table: torch.Tensor, seq_lens: torch.Tensor, page_refs: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
                   page_size: int = 64, workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Sequence ``dst[k]`` becomes a copy of sequence ``src[k]`` (int32 [n]), sharing its pages; all pairs
    read the state before the call. The last of several pairs with one target counts; pairs with a negative
    sequence are skipped."""
    b, width, stride = _table(page_table, seq_lens)
    pages = _refs(page_refs)
    n = _pairs(src, dst)
    dev = page_table.get_device()
    _same_device(dev, seq_lens, page_refs, src, dst, _status(dev_status))
    ws, ws_bytes = _workspace(workspace, pages_workspace_size(b, width, pages, n), dev, stream)
    _call("nvfp4_mla_fork_sequences", dev, page_table.data_ptr(), stride, width, seq_lens.data_ptr(), b, page_refs.data_ptr(),
          pages, page_size, src.data_ptr(), dst.data_ptr(), n, ws.data_ptr(), ws_bytes, _ptr(dev_status), _stream_of(dev, stream))


def resize_sequences(caches: Sequence[torch.Tensor], page_table: torch.Tensor, seq_lens: torch.Tensor, page_refs: torch.Tensor,
                     new_lens: torch.Tensor, max_new: int = 0, page_size: int = 64, slots: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Give each sequence the length ``new_lens[b]`` (int32 [batch]): pages are given back (0 frees a
    sequence) or taken, a shared partly filled last page is copied before its sequence grows into it (in every
    cache; ``caches`` may be empty; where all its holders grow at once, every one of them takes a page).
    Returns the slots of the first ``max_new`` new tokens of each sequence, int64 [batch, max_new], -1 where
    there is none: the slot_mapping of their append. With too few free pages no sequence grows
    (DEV_PAGES_EXHAUSTED)."""
    b, width, stride = _table(page_table, seq_lens)
    pages = _refs(page_refs)
    _need(new_lens.dtype == torch.int32 and new_lens.dim() == 1 and new_lens.shape[0] == b and new_lens.is_contiguous(),
          "new_lens int32 [batch] contiguous")
    _need(max_new >= 0, "max_new >= 0")
    dev = page_table.get_device()
    arr, num, _, rec, _ = _pool(caches, pages, page_size, dev)
    _same_device(dev, seq_lens, page_refs, new_lens, slots, _status(dev_status))
    if slots is None:
        slots = _empty((b, max_new), torch.int64, dev, stream)
    else:
        _need(slots.dtype == torch.int64 and slots.is_contiguous() and slots.shape == (b, max_new), "slots int64 [batch, max_new]")
    ws, ws_bytes = _workspace(workspace, pages_workspace_size(b, width, pages), dev, stream)
    _call("nvfp4_mla_resize_sequences", dev, page_table.data_ptr(), stride, width, seq_lens.data_ptr(), new_lens.data_ptr(), b,
          page_refs.data_ptr(), pages, page_size, arr, num, rec, slots.data_ptr(), max_new, ws.data_ptr(), ws_bytes,
          _ptr(dev_status), _stream_of(dev, stream))
    return slots


def compact_pages(caches: Sequence[torch.Tensor], page_table: torch.Tensor, seq_lens: torch.Tensor, page_refs: torch.Tensor,
                  page_size: int = 64, table_out: Optional[torch.Tensor] = None, refs_out: Optional[torch.Tensor] = None,
                  page_map: Optional[torch.Tensor] = None, live: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Move the pages in use to the front of the pool, in every cache. Returns (table, counts, page_map, live):
    the new table and counts (in place unless ``table_out`` / ``refs_out`` are given), the new page of every
    old one (-1: free), and the number of pages in use (int32 [1])."""
    b, width, stride = _table(page_table, seq_lens)
    pages = _refs(page_refs)
    table_out = page_table if table_out is None else table_out
    refs_out = page_refs if refs_out is None else refs_out
    ostride = stride
    if table_out is not page_table:
        ob, ow, ostride = _table(table_out, seq_lens, "table_out")
        _need(ob == b and ow == width, "table_out, refs_out: as page_table, page_refs")
    if refs_out is not page_refs:
        _need(_refs(refs_out) == pages, "table_out, refs_out: as page_table, page_refs")
    dev = page_table.get_device()
    arr, num, _, rec, _ = _pool(caches, pages, page_size, dev)
    _same_device(dev, seq_lens, page_refs, table_out, refs_out, page_map, live, _status(dev_status))
    if page_map is None:
        page_map = _empty((pages,), torch.int32, dev, stream)
    else:
        _need(page_map.dtype == torch.int32 and page_map.is_contiguous() and page_map.shape == (pages,), "page_map int32 [num_pages]")
    if live is None:
        live = _empty((1,), torch.int32, dev, stream)
    else:
        _need(live.dtype == torch.int32 and live.shape == (1,), "live int32 [1]")
    ws, ws_bytes = _workspace(workspace, pages_workspace_size(b, width, pages), dev, stream)
    _call("nvfp4_mla_compact_pages", dev, arr, num, rec, page_table.data_ptr(), stride, table_out.data_ptr(), ostride, width,
          seq_lens.data_ptr(), b, page_refs.data_ptr(), refs_out.data_ptr(), pages, page_size, page_map.data_ptr(), live.data_ptr(),
          ws.data_ptr(), ws_bytes, _ptr(dev_status), _stream_of(dev, stream))
    return table_out, refs_out, page_map, live
