"""The decode-step operators around the GEMMs: the paged key-value cache and
its attention, the experts' products, and token log probabilities.

Marshalling over the C ABI like the rest of the package: the arguments are
checked, packed into the C structs of ``include/wsm.h`` and handed to the
library's kernels.  Outputs and scratch come from torch's allocator on the
call's stream, so calls on other streams and captured graphs share nothing.
Tensors must lie on one device; it need not be the current one.

A call's time on the host is the whole cost of the smallest ones, so each
asks its tensors for what it needs once and checks it in one expression;
only when that fails does a second, slower pass find out what to say.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

import weight_streaming_megakernel_b200 as _wsm

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
_E4M3 = torch.float8_e4m3fn
_ROW_TYPES = (torch.bfloat16, torch.float16)
_LOGIT_TYPES = (torch.float32, torch.bfloat16, torch.float16)
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_MOST_TOP = 32
_MOST_INT = 2 ** 31 - 1

# wsm_kv_cache, wsm_kv_rows, wsm_attention, wsm_experts, wsm_logprobs
_CACHE = struct.Struct("@2P6qq4i2f")
_ROWS = struct.Struct("@2P4qP2i")
_ATTENTION = struct.Struct("@5P5qPN5if")
_EXPERTS = struct.Struct("@5P4qPN6i")
_LOGPROBS = struct.Struct("@6Pq4i")

_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns, row by row."""

    logprob: torch.Tensor       # [rows] fp32
    entropy: torch.Tensor       # [rows] fp32
    top_ids: torch.Tensor       # [rows, top] int64
    top_logprobs: torch.Tensor  # [rows, top] fp32


def _elsewhere(op, device: int, stream, *args, **kwargs):
    """`op` on a device other than the current one, or on a given stream (a
    torch stream or a raw handle), which is made current around the call so
    that outputs and scratch are allocated for it."""
    with torch.cuda.device(device):
        if stream is None:
            return op(*args, **kwargs)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream.device.index != device:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{device}")
        with torch.cuda.stream(stream):
            return op(*args, **kwargs)


def _refuse(device: int, *tensors):
    """What is wrong with a call's tensors: for each (name, tensor, shape with
    None for any size, types, contiguous in all dimensions).  Always raises."""
    for name, t, shape, types, whole in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
        if t.dtype not in types:
            raise TypeError(f"{name} must be {' or '.join(map(str, types))}, got {t.dtype}")
        if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
            raise ValueError(f"{name} must be [{', '.join('any' if n is None else str(n) for n in shape)}], "
                             f"got {list(t.shape)}")
        if whole and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")
    raise ValueError("the tensors do not fit one another")


def _shape(t, dims):
    """A tensor's shape where it has `dims` dimensions, else Nones."""
    return tuple(t.shape) if isinstance(t, torch.Tensor) and t.dim() == dims else (None,) * dims


def _types_of(t, types):
    """The types that go with `t`'s."""
    return (t.dtype,) if isinstance(t, torch.Tensor) and t.dtype in types else types


def paged_cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       slots: torch.Tensor, *, k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Write new tokens' keys and values into their slots of a paged cache.

    k, v: [tokens, kv_heads, head_dim] bf16 or fp16, any strides that are
    multiples of 16 bytes (slices of a fused qkv projection).  k_cache,
    v_cache: [pages, page_size, kv_heads, head_dim], of the same type or
    float8_e4m3fn (then value / scale is stored), in any order of the first
    three dimensions.  slots: [tokens] int64, page * page_size + place in the
    page; negative: the row is skipped.  Slots of one call must differ.
    """
    device = -1
    try:
        device = k.get_device()
        dtype, cache_dtype = k.dtype, k_cache.dtype
        tokens, heads, dim = shape = k.shape
        pages, page, cache_heads, cache_dim = cache_shape = k_cache.shape
        k0, k1, k2 = k.stride()
        v0, v1, v2 = v.stride()
        kc0, kc1, kc2, kc3 = k_cache.stride()
        vc0, vc1, vc2, vc3 = v_cache.stride()
        (n,) = slots.shape
        fits = (device >= 0 and device == v.get_device() == k_cache.get_device() == v_cache.get_device()
                == slots.get_device() and dtype in _ROW_TYPES and dtype is v.dtype and v_cache.dtype is cache_dtype
                and (cache_dtype is dtype or cache_dtype is _E4M3) and slots.dtype is _I64 and n == tokens
                and cache_heads == heads and cache_dim == dim and v.shape == shape and v_cache.shape == cache_shape
                and slots.is_contiguous() and (dim == 1 or k2 == v2 == kc3 == vc3 == 1))
    except (AttributeError, ValueError, TypeError):
        fits = False
    if not fits:
        tokens, heads, dim = _shape(k, 3)
        pages, page = _shape(k_cache, 4)[:2]
        one = _types_of(k, _ROW_TYPES)
        cached = _types_of(k_cache, one + (_E4M3,))
        _refuse(device, ("k", k, (None,) * 3, _ROW_TYPES, False), ("v", v, (tokens, heads, dim), one, False),
                ("k_cache", k_cache, (None, None, heads, dim), one + (_E4M3,), False),
                ("v_cache", v_cache, (pages, page, heads, dim), cached, False), ("slots", slots, (tokens,), (_I64,), True))
    if stream is not None or device != _current_device():
        return _elsewhere(paged_cache_append, device, stream, k, v, k_cache, v_cache, slots, k_scale=k_scale, v_scale=v_scale)
    cache = _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), kc0, kc1, kc2, vc0, vc1, vc2, pages, page, heads, dim,
                        _DTYPES[cache_dtype], k_scale, v_scale)
    rows = _ROWS.pack(k.data_ptr(), v.data_ptr(), k0, k1, v0, v1, slots.data_ptr(), tokens, _DTYPES[dtype])
    code = _wsm.lib().wsm_paged_cache_append(cache, rows, _current_stream(device))
    if code:
        _wsm._check(code, "wsm_paged_cache_append")


@functools.lru_cache(maxsize=4096)
def _attention_bytes(device: int, batch: int, head_dim: int, code: int, max_tokens: int, window: int) -> int:
    n = ctypes.c_size_t(0)
    _wsm._check(_wsm.lib().wsm_paged_attention_workspace(batch, head_dim, code, max_tokens, window, ctypes.byref(n)),
                "wsm_paged_attention_workspace")
    return n.value


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    lengths: torch.Tensor, out: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                    window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0,
                    lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one new token of each sequence over a paged cache.

    q: [batch, heads, head_dim] bf16 or fp16 (heads a multiple of the cache's
    kv_heads; head_dim 64, 96, 128 or 256); the cache as in
    paged_cache_append, with the new tokens in it.  block_table: [batch,
    pages of the longest] int32; lengths: [batch] int32 tokens of each
    sequence, the new one included, 0 for an idle row (zeros come out).
    scale: default head_dim ** -0.5.  window > 0: the last `window` tokens
    only.  lse: optional [batch, heads] fp32 buffer for the logarithm of the
    softmax's sum.  Returns out, like q (by default a new contiguous tensor).
    """
    device = -1
    try:
        device = q.get_device()
        dtype, cache_dtype = q.dtype, k_cache.dtype
        batch, heads, dim = shape = q.shape
        pages, page, kv_heads, cache_dim = cache_shape = k_cache.shape
        q0, q1, q2 = q.stride()
        k0, k1, k2, k3 = k_cache.stride()
        v0, v1, v2, v3 = v_cache.stride()
        table_rows, max_pages = block_table.shape
        t0, t1 = block_table.stride()
        (n,) = lengths.shape
        fits = (device >= 0 and device == k_cache.get_device() == v_cache.get_device() == block_table.get_device()
                == lengths.get_device() and dtype in _ROW_TYPES and v_cache.dtype is cache_dtype
                and (cache_dtype is dtype or cache_dtype is _E4M3) and block_table.dtype is lengths.dtype is _I32
                and batch == table_rows == n and cache_dim == dim and v_cache.shape == cache_shape
                and (max_pages <= 1 or t1 == 1) and lengths.is_contiguous() and (dim == 1 or q2 == k3 == v3 == 1)
                and (lse is None or (lse.get_device() == device and lse.dtype is _F32 and lse.shape == (batch, heads)
                                     and lse.is_contiguous()))
                and (out is None or (out.get_device() == device and out.dtype is dtype and out.shape == shape
                                     and out.stride(2) == 1)))
    except (AttributeError, ValueError, TypeError):
        fits = False
    if not fits:
        batch, heads, dim = _shape(q, 3)
        one = _types_of(q, _ROW_TYPES)
        more = [] if lse is None else [("lse", lse, (batch, heads), (_F32,), True)]
        more += [] if out is None else [("out", out, (batch, heads, dim), one, False)]
        pages, page, kv_heads = _shape(k_cache, 4)[:3]
        _refuse(device, ("q", q, (None,) * 3, _ROW_TYPES, False),
                ("k_cache", k_cache, (None, None, None, dim), one + (_E4M3,), False),
                ("v_cache", v_cache, (pages, page, kv_heads, dim), _types_of(k_cache, one + (_E4M3,)), False),
                ("block_table", block_table, (batch, None), (_I32,), False), ("lengths", lengths, (batch,), (_I32,), True), *more)
    if stream is not None or device != _current_device():
        return _elsewhere(paged_attention, device, stream, q, k_cache, v_cache, block_table, lengths, out, scale=scale,
                          window=window, k_scale=k_scale, v_scale=v_scale, lse=lse)
    if window > _MOST_INT:
        window = _MOST_INT                              # (more than any sequence)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        o0, o1 = heads * dim, dim
    else:
        o0, o1, _ = out.stride()
    code = _DTYPES[cache_dtype]
    n = _attention_bytes(device, batch, dim, code, max_pages * page, window)
    ws = q.new_empty(n, dtype=torch.uint8) if n else None
    cache = _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k0, k1, k2, v0, v1, v2, pages, page, kv_heads, dim, code,
                        k_scale, v_scale)
    args = _ATTENTION.pack(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), block_table.data_ptr(),
                           lengths.data_ptr(), q0, q1, o0, o1, t0, ws.data_ptr() if n else 0, n, batch, heads, max_pages,
                           window, _DTYPES[dtype], dim ** -0.5 if scale is None else scale)
    code = _wsm.lib().wsm_paged_attention(cache, args, _current_stream(device))
    if code:
        _wsm._check(code, "wsm_paged_attention")
    return out


@functools.lru_cache(maxsize=4096)
def _experts_bytes(device: int, rows: int, experts: int) -> int:
    n = _wsm.lib().wsm_expert_gemm_workspace_bytes(rows, experts)
    if n == 0:
        raise _wsm.WsmError(_wsm.WSM_ERR_UNSUPPORTED, "wsm_expert_gemm_workspace_bytes", _wsm.last_error())
    return n


def expert_gemm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                epilogue: int = 0, row_scale: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Products grouped by expert: y[r] = x[r] @ w[e].T for the rows
    offsets[e] <= r < offsets[e + 1] of expert e; returns y.

    x: [rows, K], w: [experts, N, K], both bf16 or both fp16; offsets:
    [experts + 1] int32 on the device.  With epilogue=EPI_SILU_MUL, w holds
    gate and up rows in alternating blocks of 8 and y is [rows, N / 2] =
    silu(gate) * up.  row_scale: [rows] fp32 factors of the results (router
    weights).  Rows outside all experts are left as they were: in a new y
    they are undefined.  y shares no memory with x or w.
    """
    device = -1
    try:
        device = x.get_device()
        dtype = x.dtype
        rows, k = x.shape
        experts, n, wk = w.shape
        x0, x1 = x.stride()
        w0, w1, w2 = w.stride()
        (marks,) = offsets.shape
        cols = n // 2 if epilogue == _wsm.EPI_SILU_MUL else n
        fits = (device >= 0 and device == w.get_device() == offsets.get_device() and dtype in _ROW_TYPES and w.dtype is dtype
                and offsets.dtype is _I32 and wk == k and marks == experts + 1 and offsets.is_contiguous()
                and (k == 1 or x1 == w2 == 1)
                and (row_scale is None or (row_scale.get_device() == device and row_scale.dtype is _F32
                                           and row_scale.shape == (rows,) and row_scale.is_contiguous()))
                and (y is None or (y.get_device() == device and y.dtype is dtype and y.shape == (rows, cols)
                                   and (cols == 1 or y.stride(1) == 1))))
    except (AttributeError, ValueError, TypeError):
        fits = False
    if not fits:
        rows, k = _shape(x, 2)
        experts, n, _ = _shape(w, 3)
        one = _types_of(x, _ROW_TYPES)
        more = [] if row_scale is None else [("row_scale", row_scale, (rows,), (_F32,), True)]
        more += [] if y is None else [("y", y, (rows, n if n is None or epilogue != _wsm.EPI_SILU_MUL else n // 2), one, False)]
        _refuse(device, ("x", x, (None, None), _ROW_TYPES, False), ("w", w, (None, None, k), one, False),
                ("offsets", offsets, (None if experts is None else experts + 1,), (_I32,), True), *more)
    if stream is not None or device != _current_device():
        return _elsewhere(expert_gemm, device, stream, x, w, offsets, y, epilogue=epilogue, row_scale=row_scale)
    if y is None:
        y, y0 = x.new_empty((rows, cols)), cols
    else:
        y0 = y.stride(0)
    nbytes = _experts_bytes(device, rows, experts)
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    args = _EXPERTS.pack(x.data_ptr(), w.data_ptr(), y.data_ptr(), offsets.data_ptr(),
                         0 if row_scale is None else row_scale.data_ptr(), x0, w0, w1, y0, ws.data_ptr(), nbytes,
                         rows, experts, n, k, epilogue, _DTYPES[dtype])
    code = _wsm.lib().wsm_expert_gemm(args, _current_stream(device))
    if code:
        _wsm._check(code, "wsm_expert_gemm")
    return y


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, top: int = 0,
                   stream=None) -> TokenLogprobs:
    """Log probabilities of given tokens, the entropy of each row's
    distribution and its `top` (at most 32, and the vocabulary) likeliest
    tokens.

    logits: [rows, vocab] fp32 (skinny_gemm's yf32), bf16 or fp16, rows any
    distance apart.  tokens: [rows] int64; a negative one asks for nothing and
    gets 0, as does every row without tokens.  Alternatives come likeliest
    first, equal ones by the lower index; places that no token with a
    probability above 0 takes hold -1 and -infinity.
    """
    device = -1
    try:
        device = logits.get_device()
        dtype = logits.dtype
        rows, vocab = logits.shape
        x0, x1 = logits.stride()
        fits = (device >= 0 and dtype in _LOGIT_TYPES and (vocab == 1 or x1 == 1)
                and (tokens is None or (tokens.get_device() == device and tokens.dtype is _I64 and tokens.shape == (rows,)
                                        and tokens.is_contiguous())))
    except (AttributeError, ValueError, TypeError):
        fits = False
    if not fits:
        more = [] if tokens is None else [("tokens", tokens, _shape(logits, 2)[:1], (_I64,), True)]
        _refuse(device, ("logits", logits, (None, None), _LOGIT_TYPES, False), *more)
    if stream is not None or device != _current_device():
        return _elsewhere(token_logprobs, device, stream, logits, tokens, top=top)
    width = top if 0 < top <= _MOST_TOP else 0          # (any other is refused below)
    logprob = logits.new_empty(rows, dtype=_F32)
    entropy = torch.empty_like(logprob)
    top_lp = logits.new_empty((rows, width), dtype=_F32)
    top_ids = logits.new_empty((rows, width), dtype=_I64)
    args = _LOGPROBS.pack(logits.data_ptr(), 0 if tokens is None else tokens.data_ptr(), logprob.data_ptr(),
                          entropy.data_ptr(), top_ids.data_ptr(), top_lp.data_ptr(), x0, rows, vocab,
                          min(top, _MOST_INT), _DTYPES[dtype])
    code = _wsm.lib().wsm_token_logprobs(args, _current_stream(device))
    if code:
        _wsm._check(code, "wsm_token_logprobs")
    return TokenLogprobs(logprob, entropy, top_ids, top_lp)


def operator_status(stream=None) -> int:
    """Synchronise the stream; 0, or an error that a decode-step operator
    recorded on the current device, on any stream: WSM_ERR_TIMEOUT for a
    device-side wait that ran out, before WSM_ERR_INVALID for an index out of
    range (last_error() says where).  That error is cleared; one of another
    kind stays for the next query, so ask until 0 for all of them."""
    code = ctypes.c_int(0)
    rc = _wsm.lib().wsm_operator_status(_wsm._stream_handle(stream), ctypes.byref(code))
    if rc not in (_wsm.WSM_OK, _wsm.WSM_ERR_INVALID, _wsm.WSM_ERR_TIMEOUT):
        raise _wsm.WsmError(rc, "wsm_operator_status", _wsm.last_error())
    return code.value
