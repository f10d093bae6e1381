"""The softmax-attention layers of a hybrid stack: a paged cache of keys and
values, what is appended to it and the attention of new tokens over it.

Argument marshalling only, like the package's other entry points; the names are
exported by the package."""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import _DTYPE, _I64x3, _ITYPE, OK, _raise, _stream_object, lib
from .hybrid import _I64x2, _launch, _packer, _status


class PagedArgs(ctypes.Structure):
    _fields_ = [
        ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
        ("dim", ctypes.c_int64), ("rows", ctypes.c_int64), ("nseq", ctypes.c_int64),
        ("io_dtype", ctypes.c_int32), ("table_type", ctypes.c_int32), ("meta_type", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_cache_stride", _I64x3), ("v_cache_stride", _I64x3),
        ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int64),
        ("kv_lens", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p), ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("q_stride", _I64x2), ("out_stride", _I64x2), ("d_status", ctypes.c_void_p),
    ]


_PAGED = _packer(PagedArgs)


def bind(L) -> None:
    """Argument types of these entry points on the loaded library."""
    p, i64 = ctypes.c_void_p, ctypes.c_int64  # structures are passed as their packed bytes
    L.ssu_paged_append.argtypes = [p, p, p, p, p, p, i64, ctypes.c_int32, p]
    L.ssu_paged_attention_workspace_size.argtypes = [p, i64, i64, p]
    L.ssu_paged_attention.argtypes = [p, ctypes.c_float, i64, i64, i64, p, p, ctypes.c_uint64, p]
    for fn in (L.ssu_paged_append, L.ssu_paged_attention_workspace_size, L.ssu_paged_attention):
        fn.restype = ctypes.c_int


def _on(stream, device):
    """What a call allocates belongs to the stream that it runs on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(_stream_object(device, stream))


def _paged_args(k_cache, v_cache, block_table, kv_lens, cu_seqlens, rows, heads, q, out, status) -> bytes:
    dtype = k_cache.dtype
    if not (k_cache.dim() == 4 and v_cache.shape == k_cache.shape):
        raise ValueError("k_cache and v_cache must be [pages, page_size, kv_heads, dim]")
    if not (dtype in _DTYPE and v_cache.dtype == dtype):
        raise ValueError("k_cache and v_cache must have the same dtype, fp16 or bf16")
    pages, page, kv_heads, dim = k_cache.shape
    ks, vs = k_cache.stride(), v_cache.stride()
    if not (ks[3] == vs[3] == 1):
        raise ValueError("the last dimension of the caches must have unit stride")
    if not (block_table.dim() == 2 and block_table.dtype in _ITYPE and block_table.is_cuda):
        raise ValueError("block_table must be an int32/int64 [sequences, pages] CUDA tensor")
    nseq, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("a sequence's entries of block_table must have unit stride")
    if not (kv_lens.shape == (nseq,) and kv_lens.dtype in _ITYPE and kv_lens.is_cuda and kv_lens.is_contiguous()):
        raise ValueError("kv_lens must be a contiguous int32/int64 [sequences] CUDA tensor")
    if cu_seqlens is not None:
        if not (cu_seqlens.shape == (nseq + 1,) and cu_seqlens.dtype == kv_lens.dtype and cu_seqlens.is_cuda
                and cu_seqlens.is_contiguous()):
            raise ValueError("cu_seqlens must be a contiguous [sequences + 1] CUDA tensor in kv_lens' dtype")
    elif rows != nseq:
        raise ValueError("without cu_seqlens every sequence has one row")
    if not (k_cache.is_cuda and v_cache.is_cuda):
        raise ValueError("all tensors must be CUDA tensors")
    qs, os = (0, 0) if q is None else q.stride(), (0, 0) if out is None else out.stride()
    return _PAGED.pack(pages, page, heads, kv_heads, dim, rows, nseq, _DTYPE[dtype], _ITYPE[block_table.dtype],
                       _ITYPE[kv_lens.dtype], 0, k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1],
                       vs[2], block_table.data_ptr(), block_table.stride(0), width, kv_lens.data_ptr(),
                       0 if cu_seqlens is None else cu_seqlens.data_ptr(), 0 if q is None else q.data_ptr(),
                       0 if out is None else out.data_ptr(), qs[0], qs[1], os[0], os[1], _status(status))


def _rows_like(name, t, rows, heads, dim, dtype):
    if not (t.shape == (rows, heads, dim) and t.dtype == dtype and t.is_cuda and t.stride(2) == 1):
        raise ValueError(f"{name} must be a [{rows}, {heads}, {dim}] CUDA tensor in the caches' dtype with unit stride along dim")


def ssu_paged_append(k_cache, v_cache, k, v, block_table, kv_lens, cu_seqlens=None, q=None, inv_freq=None,
                     interleaved: bool = False, q_out=None, status=None, stream=None) -> Optional[torch.Tensor]:
    """Append new tokens' keys and values to a paged cache, turned by their
    position (``ssu_paged_append`` in ``include/ssu.h``).

    ``k_cache`` and ``v_cache`` are ``[pages, page_size, kv_heads, dim]``, k and v
    ``[rows, kv_heads, dim]``, q ``[rows, heads, dim]`` (slices of a fused
    projection are fine); ``block_table`` ``[sequences, pages of the longest]``;
    ``kv_lens`` ``[sequences]`` counts the new tokens too; ``cu_seqlens`` are the
    bounds of the sequences' rows (default: one row each).  ``inv_freq``, fp32
    ``[rotary / 2]``, holds the angles per position of the pairs ``(j, j + rotary
    / 2)``, or ``(2 j, 2 j + 1)`` if ``interleaved``; None turns nothing.  Returns
    the turned q (``q_out``, which may be q; default: a new tensor), None
    without q."""
    if not (k.dim() == 3 and v.dim() == 3 and k_cache.dim() == 4):
        raise ValueError("k and v are [rows, kv_heads, dim], the caches [pages, page_size, kv_heads, dim]")
    rows, dtype = k.shape[0], k_cache.dtype
    kv_heads, dim = k_cache.shape[2:]
    _rows_like("k", k, rows, kv_heads, dim, dtype)
    _rows_like("v", v, rows, kv_heads, dim, dtype)
    heads = kv_heads
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q is [rows, heads, dim]")
        heads = q.shape[1]
        _rows_like("q", q, rows, heads, dim, dtype)
        if q_out is None:
            with _on(stream, q.device):
                q_out = torch.empty((rows, heads, dim), dtype=dtype, device=q.device)
        else:
            _rows_like("q_out", q_out, rows, heads, dim, dtype)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    rotary = 0
    if inv_freq is not None:
        if not (inv_freq.dtype == torch.float32 and inv_freq.dim() == 1 and inv_freq.is_cuda and inv_freq.is_contiguous()
                and inv_freq.numel() > 0):
            raise ValueError("inv_freq must be a contiguous fp32 [rotary / 2] CUDA tensor")
        rotary = 2 * inv_freq.numel()
    a = _paged_args(k_cache, v_cache, block_table, kv_lens, cu_seqlens, rows, heads, q, q_out, status)
    ks, vs = k.stride(), v.stride()
    _launch(lib().ssu_paged_append, k_cache.get_device(), stream, a, k.data_ptr(), _I64x2(ks[0], ks[1]), v.data_ptr(),
            _I64x2(vs[0], vs[1]), None if inv_freq is None else inv_freq.data_ptr(), rotary, int(bool(interleaved)))
    return q_out


def ssu_paged_attention(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, scale: Optional[float] = None,
                        window: int = 0, max_seqlen: Optional[int] = None, max_kv_len: Optional[int] = None, out=None,
                        return_lse: bool = False, status=None, stream=None):
    """Attention of new tokens over a paged cache that holds them already
    (``ssu_paged_attention`` in ``include/ssu.h``): single tokens, drafts,
    chunks of prompts, or all of them in one call.

    q is ``[rows, heads, dim]``; the caches, ``block_table``, ``kv_lens`` and
    ``cu_seqlens`` are those of :func:`ssu_paged_append`.  A token sees the keys
    up to its own, with ``window`` only the last ``window`` of them.  ``scale``
    defaults to ``dim ** -0.5``.  Pass ``max_seqlen`` and ``max_kv_len`` (the most
    new tokens and the most tokens of a sequence) where they are known on the
    host; they only steer how the work is split.  Returns out ``[rows, heads,
    dim]``, with ``return_lse`` (out, lse), lse fp32 ``[rows, heads]``."""
    if not (q.dim() == 3 and k_cache.dim() == 4):
        raise ValueError("q is [rows, heads, dim], the caches [pages, page_size, kv_heads, dim]")
    rows, heads, dim = q.shape[0], q.shape[1], k_cache.shape[3]
    _rows_like("q", q, rows, heads, dim, k_cache.dtype)
    if out is not None:
        _rows_like("out", out, rows, heads, dim, k_cache.dtype)
    L, lse = lib(), None
    seqlen, kv_len = 0 if max_seqlen is None else max_seqlen, 0 if max_kv_len is None else max_kv_len
    with _on(stream, q.device):
        if out is None:
            out = torch.empty((rows, heads, dim), dtype=q.dtype, device=q.device)
        if return_lse:
            lse = torch.empty((rows, heads), dtype=torch.float32, device=q.device)
        a = _paged_args(k_cache, v_cache, block_table, kv_lens, cu_seqlens, rows, heads, q, out, status)
        nbytes = ctypes.c_uint64(0)
        rc = L.ssu_paged_attention_workspace_size(a, seqlen, kv_len, ctypes.byref(nbytes))
        if rc != OK:
            _raise(rc)
        # a block of the caching allocator for this call alone (in a capture, of the graph's own pool)
        ws = torch.empty(nbytes.value, dtype=torch.uint8, device=q.device) if nbytes.value else None
    _launch(L.ssu_paged_attention, k_cache.get_device(), stream, a, dim ** -0.5 if scale is None else scale, window, seqlen,
            kv_len, None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), nbytes.value)
    return (out, lse) if return_lse else out
