"""Binding of the calls around the latent attention (``include/nvfp4_mla.h``, "Heads and latents"): the
query into the latent space and the output back out of it (the absorbed form), records in pages expanded
into per-head keys and values, and the attention of chunks over them (the expanded form). Argument
marshalling only, as in the package's other calls.

``kv_b`` is the latent's up-projection, bf16 [h, 256, 512] with inner stride 1: per head 128 rows for the
key, then 128 for the value. Tokens and heads of the inputs may have any strides that are multiples of 8
elements. The calls work on the tensors' own device, whichever is current, and on ``stream`` (default: that
device's current stream)."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import D_NOPE, D_QK, D_ROPE, _check, _need, _ptr, _record_code, load
from .paged import _empty, _same_device, _status, _stream_of, _workspace

D_HEAD_NOPE, D_HEAD_V = 128, 128
D_HEAD_QK, D_HEAD_KV = D_HEAD_NOPE + D_ROPE, D_HEAD_NOPE + D_HEAD_V

# These calls are small next to a layer's others, so their host time counts: checks read each property of a tensor once, and
# messages are put together only where they are raised (one token with `out` given: 10.2 -> 7.6 us on the host, 3.6 of them in C).
_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
_calls = {}


def _call(name: str, dev: int, *args) -> None:
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = getattr(load(), name)
    if torch._C._cuda_getDevice() == dev:   # (read here: a build of torch without CUDA has no such name, and the package imports there too)
        st = f(*args)
    else:
        with torch.cuda.device(dev):
            st = f(*args)
    if st:
        _check(name, st)


def _strides(t: torch.Tensor, width: int, name: str):
    """(tokens, heads, token stride, head stride) of a bf16 [tokens, heads, width] tensor"""
    if t.dtype is _BF16 and t.dim() == 3:
        tokens, heads, d = t.shape
        a, b, c = t.stride()
        if d == width and (c == 1 or tokens * heads == 0):
            return tokens, heads, a, b
    raise ValueError(f"{name} bf16 [T,h,{width}], inner stride 1")


def _weights(kv_b: torch.Tensor, h: int):
    """(row stride, head stride)"""
    if kv_b.dtype is _BF16 and kv_b.dim() == 3 and kv_b.shape == (h, D_HEAD_KV, D_NOPE):
        a, b, c = kv_b.stride()
        if c == 1:
            return b, a
    raise ValueError("kv_b bf16 [h,256,512], inner stride 1, with as many heads as the other tensors")


def _result(out: Optional[torch.Tensor], shape, dtype, dev: int, stream, name: str) -> torch.Tensor:
    if out is None:
        return _empty(shape, dtype, dev, stream)
    if out.dtype is not dtype or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"{name} {dtype} {list(shape)} contiguous")
    return out


def _starts(t: torch.Tensor, name: str) -> int:
    """batch of an int32 [batch + 1] tensor"""
    if t.dtype is not _I32 or t.dim() != 1 or t.shape[0] < 1 or not t.is_contiguous():
        raise ValueError(name + " int32 [batch + 1] contiguous")
    return t.shape[0] - 1


@functools.lru_cache(maxsize=1)
def ragged_workspace_size() -> int:
    """Workspace bytes of ragged_mla_attention, whatever the sizes."""
    n = ctypes.c_size_t(0)
    _check("nvfp4_ragged_mla_attention_workspace_size", load().nvfp4_ragged_mla_attention_workspace_size(ctypes.byref(n)))
    return int(n.value)


def mla_absorb_query(q: torch.Tensor, kv_b: torch.Tensor, positions: Optional[torch.Tensor] = None, cos_table: Optional[torch.Tensor] = None,
                     sin_table: Optional[torch.Tensor] = None, rotate_half: bool = True, out: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The query of the latent attention: q bf16 [T, h, 192] (128 NoPE dims, 64 RoPE dims) -> bf16 [T, h, 576],
    ``q[t, h, :128] @ kv_b[h, :128]`` beside the RoPE dims, rotated by ``positions`` (int64 [T]) with
    ``cos_table`` / ``sin_table`` (fp32 [P, 32]), pairs (f, f+32) when ``rotate_half`` else (2f, 2f+1); without
    ``positions`` they are copied. The result is what paged_mla_decode and sparse_mla_decode take, viewed as
    [B, s_q, h, 576]."""
    T, h, ts, hs = _strides(q, D_HEAD_QK, "q")
    ws, wh = _weights(kv_b, h)
    rows = 0
    if positions is None:
        _need(cos_table is None and sin_table is None, "cos_table and sin_table go with positions")
    else:
        if positions.dtype is not _I64 or positions.shape != (T,) or not positions.is_contiguous():
            raise ValueError("positions int64 [T] contiguous")
        if cos_table is None or sin_table is None or cos_table.dtype is not _F32 or sin_table.dtype is not _F32 or cos_table.dim() != 2:
            raise ValueError("cos_table / sin_table fp32 [P,32] contiguous")
        rows, d = cos_table.shape
        if d != 32 or sin_table.shape != (rows, d) or not cos_table.is_contiguous() or not sin_table.is_contiguous():
            raise ValueError("cos_table / sin_table fp32 [P,32] contiguous")
    dev = q.get_device()   # -1 for a CPU tensor
    _same_device(dev, kv_b, positions, cos_table, sin_table, out, _status(dev_status))
    out = _result(out, (T, h, D_QK), _BF16, dev, stream, "out")
    _call("nvfp4_mla_absorb_query", dev, q.data_ptr(), ts, hs, kv_b.data_ptr(), ws, wh, _ptr(positions), _ptr(cos_table), _ptr(sin_table), rows,
          1 if rotate_half else 0, T, h, out.data_ptr(), _ptr(dev_status), _stream_of(dev, stream))
    return out


def mla_project_values(latent: torch.Tensor, kv_b: torch.Tensor, out: Optional[torch.Tensor] = None,
                       dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The heads' outputs from the latent attention's: latent bf16 [T, h, 512] -> bf16 [T, h, 128],
    ``kv_b[h, 128:] @ latent[t, h]``."""
    T, h, ts, hs = _strides(latent, D_NOPE, "latent")
    ws, wh = _weights(kv_b, h)
    dev = latent.get_device()
    _same_device(dev, kv_b, out, _status(dev_status))
    out = _result(out, (T, h, D_HEAD_V), _BF16, dev, stream, "out")
    _call("nvfp4_mla_project_values", dev, latent.data_ptr(), ts, hs, kv_b.data_ptr(), ws, wh, T, h, out.data_ptr(), _ptr(dev_status),
          _stream_of(dev, stream))
    return out


def paged_mla_expand(cache: torch.Tensor, page_table: torch.Tensor, cu_seqlens: torch.Tensor, kv_b: torch.Tensor, num_rows: int,
                     page_size: int = 64, kv: Optional[torch.Tensor] = None, k_pe: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None, block_scales: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-head keys and values of the sequences' first ``cu_seqlens[b + 1] - cu_seqlens[b]`` tokens (int32
    [batch + 1], on the device), read from their records in pages (cache uint8 [num_pages * page_size, 352|432])
    and packed one sequence behind the other: kv bf16 [num_rows, h, 256] (128 dims of the key, 128 of the value)
    and k_pe bf16 [num_rows, 64], the RoPE dims that all heads share. Rows from ``cu_seqlens[batch]`` on are left
    as they were. ``block_scales``: the cache holds 352-byte records with their scales in block order."""
    _need(kv_b.dim() == 3, "kv_b bf16 [h,256,512]")
    h = kv_b.shape[0]
    ws, wh = _weights(kv_b, h)
    _need(num_rows >= 0, "num_rows >= 0")
    batch = _starts(cu_seqlens, "cu_seqlens")
    if page_table.dtype is not _I32 or page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError("page_table int32 [batch, max_pages], inner stride 1")
    width = page_table.shape[1]
    stride, inner = page_table.stride()
    _need(width <= 1 or inner == 1, "page_table int32 [batch, max_pages], inner stride 1")
    if batch <= 1:
        stride = max(width, 1)
    _need(stride >= width, "page_table rows overlap")
    if cache.dtype is not _U8 or cache.dim() != 2 or not cache.is_contiguous() or cache.shape[1] not in (352, 432):
        raise ValueError("cache uint8 [num_slots, 352|432] contiguous")
    _need(page_size > 0, "page_size is a power of two")
    code = _record_code(cache, block_scales)
    dev = cache.get_device()
    _same_device(dev, page_table, cu_seqlens, kv_b, kv, k_pe, _status(dev_status))
    kv = _result(kv, (num_rows, h, D_HEAD_KV), _BF16, dev, stream, "kv")
    k_pe = _result(k_pe, (num_rows, D_ROPE), _BF16, dev, stream, "k_pe")
    _call("nvfp4_paged_mla_expand", dev, cache.data_ptr(), cache.shape[0] // page_size, page_size, code, page_table.data_ptr(), stride, width,
          cu_seqlens.data_ptr(), batch, kv_b.data_ptr(), ws, wh, h, kv.data_ptr(), k_pe.data_ptr(), num_rows, _ptr(dev_status),
          _stream_of(dev, stream))
    return kv, k_pe


def ragged_mla_attention(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                         sm_scale: float, attn_sink: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         dev_status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention of the last tokens of each sequence over all its tokens, in the expanded form: q bf16
    [Tq, h, 192] (rotated RoPE dims last), kv bf16 [Tk, h, 256] and k_pe bf16 [Tk, 64] as from paged_mla_expand, or from
    a projection of unquantized latents. Sequence b has the queries ``cu_seqlens_q[b]`` to ``cu_seqlens_q[b + 1]``
    (int32 [batch + 1], on the device) and the keys ``cu_seqlens_k[b]`` to ``cu_seqlens_k[b + 1]``; its last query sees all of
    them, the one before it one fewer, and so on. Returns (out bf16 [Tq, h, 128], lse fp32 [Tq, h]); a query without
    a visible key gets out = 0, lse = -inf, rows from ``cu_seqlens_q[batch]`` on are left as they were. The kernel is chosen by the
    average rows and keys of a sequence (Tq / batch, Tk / batch): padding sequences, or tensors far larger than the batch, may cost long
    chunks some of their speed."""
    Tq, h, qt, qh = _strides(q, D_HEAD_QK, "q")
    Tk, hk, kt, kh = _strides(kv, D_HEAD_KV, "kv")
    _need(hk == h, "q and kv disagree about the heads")
    if k_pe.dtype is not _BF16 or k_pe.shape != (Tk, D_ROPE) or (k_pe.stride(1) != 1 and Tk > 0):
        raise ValueError("k_pe bf16 [Tk,64], inner stride 1")
    batch = _starts(cu_seqlens_q, "cu_seqlens_q")
    _need(_starts(cu_seqlens_k, "cu_seqlens_k") == batch, "cu_seqlens_q and cu_seqlens_k differ in length")
    if attn_sink is not None:
        _need(attn_sink.dtype is _F32 and attn_sink.numel() == h and attn_sink.is_contiguous(), "attn_sink fp32 [h]")
    dev = q.get_device()
    _same_device(dev, kv, k_pe, cu_seqlens_q, cu_seqlens_k, attn_sink, out, lse, _status(dev_status))
    out = _result(out, (Tq, h, D_HEAD_V), _BF16, dev, stream, "out")
    lse = _result(lse, (Tq, h), _F32, dev, stream, "lse")
    ws, ws_bytes = _workspace(workspace, ragged_workspace_size(), dev, stream)
    _call("nvfp4_ragged_mla_attention", dev, q.data_ptr(), qt, qh, Tq, kv.data_ptr(), kt, kh, k_pe.data_ptr(), k_pe.stride(0), Tk,
          cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), batch, h, float(sm_scale), _ptr(attn_sink), out.data_ptr(), lse.data_ptr(),
          ws.data_ptr(), ws_bytes, _ptr(dev_status), _stream_of(dev, stream))
    return out, lse
