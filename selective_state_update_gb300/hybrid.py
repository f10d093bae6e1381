"""The operators around the state update in a hybrid stack: linear attention
with a decay for each head on the same slot pools, the residual-adding RMS norm
with an 8-bit output, and the log probabilities of given tokens.

Argument marshalling only, like the package's other entry points; the names are
exported by the package."""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import _DTYPE, _I64x3, _ITYPE, _raise, _stream, _stream_object, _table, OK, SLOTS_STRIDED, SlotTable, lib

_I64x2 = ctypes.c_int64 * 2

NORM_PLAIN, NORM_ROW, NORM_BLOCK = 0, 1, 2  # SSU_NORM_*
NORM_BLOCK_COLUMNS = 128
MAX_TOP_K = 32
_NORM_FORMAT = {"none": NORM_PLAIN, "row": NORM_ROW, "block": NORM_BLOCK}


class LinattnArgs(ctypes.Structure):
    _fields_ = [
        ("slots", ctypes.c_int64), ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64), ("dim", ctypes.c_int64),
        ("dstate", ctypes.c_int64), ("rows", ctypes.c_int64),
        ("io_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reserved0", ctypes.c_int32), ("pad_slot_id", ctypes.c_int64),
        ("state", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("log_decay", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("q_stride", _I64x2), ("k_stride", _I64x2), ("v_stride", _I64x2), ("out_stride", _I64x2),
        ("d_status", ctypes.c_void_p),
    ]


class NormArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("hidden", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32), ("format", ctypes.c_int32), ("eps", ctypes.c_float),
        ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("weight", ctypes.c_void_p),
        ("residual_out", ctypes.c_void_p), ("y", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64), ("residual_out_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64),
    ]


class LogprobArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("row_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("token_type", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("logits", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("logprobs", ctypes.c_void_p),
        ("entropy", ctypes.c_void_p), ("top_ids", ctypes.c_void_p), ("top_logprobs", ctypes.c_void_p),
        ("d_status", ctypes.c_void_p),
    ]


def _packer(cls) -> struct.Struct:
    """The C layout of a ctypes structure for one struct.pack call: filling the
    structure field by field costs more than some of the kernels take."""
    code = {ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_void_p: "Q", _I64x2: "2q",
            _I64x3: "3q"}
    return struct.Struct("@" + "".join(code[f[1]] for f in cls._fields_))


_LINATTN, _NORM, _LOGPROB, _SLOTS = (_packer(c) for c in (LinattnArgs, NormArgs, LogprobArgs, SlotTable))


def bind(L) -> None:
    """Argument types of these entry points on the loaded library."""
    p = ctypes.c_void_p  # structures are passed as their packed bytes
    L.ssu_linear_attention_step.argtypes = [p, p, p, p]
    L.ssu_linear_attention_workspace_size.argtypes = [p, ctypes.c_int64, ctypes.c_int64, p]
    L.ssu_linear_attention_prefill.argtypes = [p, ctypes.c_int64, p, ctypes.c_int32, ctypes.c_int64, p, p, p,
                                               ctypes.c_uint64, p]
    L.ssu_add_rmsnorm.argtypes = [p, p]
    L.ssu_token_logprobs.argtypes = [p, p]
    for fn in (L.ssu_linear_attention_step, L.ssu_linear_attention_workspace_size, L.ssu_linear_attention_prefill,
               L.ssu_add_rmsnorm, L.ssu_token_logprobs):
        fn.restype = ctypes.c_int


def _launch(fn, device: int, stream, *args) -> None:
    """fn(*args, stream) with the operands' device current; raises what it reports."""
    handle = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == device:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != OK:
        _raise(rc)


def _slots(t: Optional[torch.Tensor]):
    """A slot table's packed structure."""
    if t is None:
        return None
    if t.dim() == 1 and t.is_cuda and t.dtype in _ITYPE:
        n, s = t.shape[0], t.stride(0)
        return _SLOTS.pack(t.data_ptr(), _ITYPE[t.dtype], SLOTS_STRIDED, s, s, (n - 1) * s + 1 if n else 0)
    return ctypes.byref(_table(t, SLOTS_STRIDED))


def _status(status: Optional[torch.Tensor]) -> int:
    if status is None:
        return 0
    if not (status.dtype == torch.int32 and status.numel() >= 1 and status.is_cuda):
        raise ValueError("status must be an int32 CUDA tensor")
    return status.data_ptr()


def _linattn_args(state, q, k, v, log_decay, scale, pad_slot_id, out, status):
    """(packed arguments, out)."""
    if not (state.dim() == 4 and state.is_contiguous()):
        raise ValueError("state must be a contiguous [slots, heads, dim, dstate] tensor")
    if not (q.dim() == 3 and k.dim() == 3 and v.dim() == 3):
        raise ValueError("q, k and v are [rows, heads, head size]")
    slots, heads, dim, dstate = state.shape
    rows, kv_heads, dtype = q.shape[0], k.shape[1], q.dtype
    if q.shape != (rows, heads, dstate):
        raise ValueError("q must be [rows, heads, dstate]")
    if k.shape != (rows, kv_heads, dstate):
        raise ValueError("k must be [rows, kv_heads, dstate]")
    if v.shape != (rows, kv_heads, dim):
        raise ValueError("v must be [rows, kv_heads, dim]")
    if not (state.dtype in _DTYPE and dtype in _DTYPE):
        raise ValueError("unsupported dtype")
    if not (k.dtype == dtype and v.dtype == dtype):
        raise ValueError("k and v must have the dtype of q")
    if out is None:
        out = torch.empty((rows, heads, dim), dtype=dtype, device=q.device)
    else:
        if not (out.shape == (rows, heads, dim) and out.dtype == dtype):
            raise ValueError("out must be [rows, heads, dim] in q's dtype")
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    if not (qs[2] == ks[2] == vs[2] == os[2] == 1):
        raise ValueError("the last dimension of q, k, v and out must have unit stride")
    if not (log_decay.dtype == torch.float32 and log_decay.shape == (heads,) and log_decay.is_contiguous()):
        raise ValueError("log_decay must be a contiguous fp32 [heads] tensor")
    if not (state.is_cuda and q.is_cuda and k.is_cuda and v.is_cuda and out.is_cuda and log_decay.is_cuda):
        raise ValueError("all tensors must be CUDA tensors")
    return _LINATTN.pack(slots, heads, kv_heads, dim, dstate, rows, _DTYPE[dtype], _DTYPE[state.dtype],
                         dstate ** -0.5 if scale is None else scale, 0, pad_slot_id, state.data_ptr(), q.data_ptr(),
                         k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), out.data_ptr(), qs[0], qs[1], ks[0], ks[1],
                         vs[0], vs[1], os[0], os[1], _status(status)), out


def ssu_linear_attention_step(state, q, k, v, log_decay, scale: Optional[float] = None, state_batch_indices=None,
                              dst_state_batch_indices=None, pad_slot_id: int = -1, out=None, status=None,
                              stream=None) -> torch.Tensor:
    """One token of linear attention per sequence (``ssu_linear_attention_step``
    in ``include/ssu.h``): S = exp(log_decay[h]) S + v k^T, out = scale S q.

    ``state`` is the slot pool ``[slots, heads, dim, dstate]``, updated in
    place; q ``[batch, heads, dstate]``, k ``[batch, kv_heads, dstate]``, v
    ``[batch, kv_heads, dim]`` (slices of a fused projection are fine),
    ``log_decay`` fp32 ``[heads]``; ``scale`` defaults to ``dstate ** -0.5``.
    Returns out ``[batch, heads, dim]`` in q's dtype."""
    a, out = _linattn_args(state, q, k, v, log_decay, scale, pad_slot_id, out, status)
    _launch(lib().ssu_linear_attention_step, state.get_device(), stream, a, _slots(state_batch_indices),
            _slots(dst_state_batch_indices))
    return out


def ssu_linear_attention_prefill(state, q, k, v, log_decay, cu_seqlens, scale: Optional[float] = None,
                                 state_batch_indices=None, dst_state_batch_indices=None, pad_slot_id: int = -1,
                                 max_seqlen: Optional[int] = None, out=None, status=None, stream=None) -> torch.Tensor:
    """Linear attention over packed prompts (``ssu_linear_attention_prefill`` in
    ``include/ssu.h``): q ``[tokens, heads, dstate]``, k and v per kv head, the
    sequences' bounds ``cu_seqlens`` ``[nseq + 1]``.

    Sequence b starts from slot ``state_batch_indices[b]`` (``pad_slot_id``:
    from zeros) and leaves its final state in slot
    ``dst_state_batch_indices[b]`` (default: the slot it started from).  Pass
    ``max_seqlen`` where it is known on the host; it only steers how the work is
    split.  Returns out ``[tokens, heads, dim]`` in q's dtype."""
    if not (cu_seqlens.dtype in _ITYPE and cu_seqlens.is_cuda and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous()
            and cu_seqlens.numel() >= 1):
        raise ValueError("cu_seqlens must be a contiguous int32/int64 [nseq + 1] CUDA tensor")
    a, out = _linattn_args(state, q, k, v, log_decay, scale, pad_slot_id, out, status)
    nseq, longest = cu_seqlens.shape[0] - 1, 0 if max_seqlen is None else max_seqlen
    nbytes = ctypes.c_uint64(0)
    L = lib()
    rc = L.ssu_linear_attention_workspace_size(a, nseq, longest, ctypes.byref(nbytes))
    if rc != OK:
        _raise(rc)
    need, ws = nbytes.value, None
    if need:
        # a block of the caching allocator for this call alone, on the stream
        # that it runs on (in a capture, of the graph's own pool): the launches of
        # another host thread's call may come between this one's
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            with torch.cuda.stream(_stream_object(q.device, stream)):
                ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    _launch(L.ssu_linear_attention_prefill, state.get_device(), stream, a, nseq, cu_seqlens.data_ptr(),
            _ITYPE[cu_seqlens.dtype], longest, _slots(state_batch_indices), _slots(dst_state_batch_indices),
            None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return out


def ssu_add_rmsnorm(x, weight, eps: float = 1e-5, residual=None, quant: str = "none", residual_out=None, out=None,
                    scales=None, stream=None):
    """RMS norm of the rows of x ``[rows, hidden]``, with the residual's
    addition before it (``ssu_add_rmsnorm`` in ``include/ssu.h``).

    ``quant`` is "none" (out in x's dtype), "row" (``float8_e4m3fn`` codes with
    one fp32 scale per row) or "block" (one per 128 columns, ``[rows,
    ceil(hidden / 128)]``).  ``residual_out`` receives x + residual; it may be
    the residual itself (default: a new tensor).  Returns (out, scales,
    residual_out); scales is None for "none", residual_out without a
    residual."""
    if not (x.dim() == 2 and x.dtype in _DTYPE and x.is_cuda and x.stride(1) == 1):
        raise ValueError("x must be a [rows, hidden] CUDA tensor with unit column stride")
    rows, hidden = x.shape
    fmt = _NORM_FORMAT.get(quant)
    if fmt is None:
        raise ValueError("quant is 'none', 'row' or 'block'")
    if not (weight.shape == (hidden,) and weight.dtype in (x.dtype, torch.float32) and weight.is_contiguous() and weight.is_cuda):
        raise ValueError("weight must be a contiguous [hidden] CUDA tensor in x's dtype or fp32")
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
    else:
        if not (residual.shape == x.shape and residual.dtype == x.dtype and residual.is_cuda and residual.stride(1) == 1):
            raise ValueError("residual must match x and have unit column stride")
        if residual_out is None:
            residual_out = torch.empty((rows, hidden), dtype=x.dtype, device=x.device)
        else:
            if not (residual_out.shape == x.shape and residual_out.dtype == x.dtype and residual_out.is_cuda
                    and residual_out.stride(1) == 1):
                raise ValueError("residual_out must match x and have unit column stride")
    y_dtype = x.dtype if fmt == NORM_PLAIN else torch.float8_e4m3fn
    if out is None:
        out = torch.empty((rows, hidden), dtype=y_dtype, device=x.device)
    else:
        if not (out.shape == x.shape and out.dtype == y_dtype and out.is_cuda and out.stride(1) == 1):
            raise ValueError(f"out must be a [rows, hidden] {y_dtype} CUDA tensor with unit column stride")
    if fmt == NORM_PLAIN:
        if scales is not None:
            raise ValueError("scales go with an 8-bit output")
    else:
        shape = (rows,) if fmt == NORM_ROW else (rows, -(-hidden // NORM_BLOCK_COLUMNS))
        if scales is None:
            scales = torch.empty(shape, dtype=torch.float32, device=x.device)
        else:
            if not (scales.shape == shape and scales.dtype == torch.float32 and scales.is_contiguous() and scales.is_cuda):
                raise ValueError(f"scales must be a contiguous fp32 CUDA tensor of shape {shape}")
    res, res_out = (0, 0) if residual is None else (residual.data_ptr(), residual_out.data_ptr())
    a = _NORM.pack(rows, hidden, _DTYPE[x.dtype], _DTYPE[weight.dtype], fmt, eps, x.data_ptr(), res, weight.data_ptr(),
                   res_out, out.data_ptr(), 0 if scales is None else scales.data_ptr(), x.stride(0),
                   0 if residual is None else residual.stride(0), 0 if residual is None else residual_out.stride(0),
                   out.stride(0))
    _launch(lib().ssu_add_rmsnorm, x.get_device(), stream, a)
    return out, scales, residual_out


def ssu_token_logprobs(logits, tokens, top_k: int = 0, status=None, stream=None):
    """Log probabilities of ``tokens`` ``[rows]`` under ``logits`` ``[rows,
    vocab]``, the rows' entropy and the ``top_k`` most likely alternatives
    (``ssu_token_logprobs`` in ``include/ssu.h``).

    Returns (logprobs ``[rows]``, entropy ``[rows]``, top_ids ``[rows, top_k]``
    in tokens' dtype, top_logprobs ``[rows, top_k]``), the floating ones fp32;
    the last two are None without ``top_k``.  Token -1 asks for none."""
    if not (logits.dim() == 2 and logits.dtype in _DTYPE and logits.is_cuda and logits.stride(1) == 1):
        raise ValueError("logits must be a [rows, vocab] CUDA tensor with unit column stride")
    rows, vocab = logits.shape
    if not (tokens.shape == (rows,) and tokens.dtype in _ITYPE and tokens.is_cuda and tokens.is_contiguous()):
        raise ValueError("tokens must be a contiguous int32/int64 [rows] CUDA tensor")
    device = logits.device
    logprobs = torch.empty(rows, dtype=torch.float32, device=device)
    entropy = torch.empty(rows, dtype=torch.float32, device=device)
    ids = top = None
    if top_k > 0:
        ids = torch.empty((rows, top_k), dtype=tokens.dtype, device=device)
        top = torch.empty((rows, top_k), dtype=torch.float32, device=device)
    a = _LOGPROB.pack(rows, vocab, logits.stride(0), _DTYPE[logits.dtype], _ITYPE[tokens.dtype], top_k, 0, logits.data_ptr(),
                      tokens.data_ptr(), logprobs.data_ptr(), entropy.data_ptr(), 0 if ids is None else ids.data_ptr(),
                      0 if top is None else top.data_ptr(), _status(status))
    _launch(lib().ssu_token_logprobs, logits.get_device(), stream, a)
    return logprobs, entropy, ids, top
