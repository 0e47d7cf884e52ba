"""The decode-step operators around the GEMMs: the paged key-value cache and
its attention, the experts' products, and token log probabilities.

Marshalling over the C ABI like the rest of the package: the arguments are
checked, packed into the C structs of ``include/wsm.h`` and handed to the
library's kernels.  Outputs and scratch come from torch's allocator on the
call's stream, so calls on other streams and captured graphs share nothing.
Tensors must lie on one device; it need not be the current one.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

import weight_streaming_megakernel_b200 as _wsm

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
_BF16, _FP16, _FP32, _E4M3 = range(4)

# wsm_kv_cache, wsm_kv_rows, wsm_attention, wsm_experts, wsm_logprobs
_CACHE = struct.Struct("@2P6qq4i2f")
_ROWS = struct.Struct("@2P4qP2i")
_ATTENTION = struct.Struct("@5P5qPN5if")
_EXPERTS = struct.Struct("@5P4qPN6i")
_LOGPROBS = struct.Struct("@6Pq4i")

_INT_MAX = 2**31 - 1


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns, row by row."""

    logprob: torch.Tensor       # [rows] fp32
    entropy: torch.Tensor       # [rows] fp32
    top_ids: torch.Tensor       # [rows, top] int64
    top_logprobs: torch.Tensor  # [rows, top] fp32


def _tensor(name, t, dims, device=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(shape)}")
    if max(shape) > _INT_MAX:
        raise ValueError(f"{name} is too large: {tuple(shape)}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return shape


def _dtype(name, t, allowed):
    code = _DTYPES.get(t.dtype, -1)
    if code not in allowed:
        raise TypeError(f"{name} cannot be {t.dtype}")
    return code


def _output(name, t, shape, device, dtype):
    """A caller's contiguous output buffer."""
    _tensor(name, t, len(shape), device, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_stream(op):
    """`op` runs on the current stream of its tensors' device.  With stream=
    (a torch stream or a raw handle) that stream is made current around the
    call, so that outputs and scratch are allocated for it; likewise a device
    other than the current one."""

    @functools.wraps(op)
    def call(first, *args, stream=None, **kwargs):
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            return op(first, *args, **kwargs)  # its own checks say what is wrong
        index = first.device.index
        if stream is None and index == torch.cuda.current_device():
            return op(first, *args, **kwargs)
        with torch.cuda.device(index):
            if stream is None:
                return op(first, *args, **kwargs)
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=first.device)
            if stream.device.index != index:
                raise ValueError(f"the stream belongs to {stream.device}, the tensors to {first.device}")
            with torch.cuda.stream(stream):
                return op(first, *args, **kwargs)

    return call


def _current(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


@functools.lru_cache(maxsize=4096)
def _attention_bytes(device_index: int, batch: int, head_dim: int) -> int:
    n = _wsm.lib().wsm_paged_attention_workspace_bytes(batch, head_dim)
    if n == 0:
        raise _wsm.WsmError(_wsm.WSM_ERR_UNSUPPORTED, "wsm_paged_attention_workspace_bytes", _wsm.last_error())
    return n


@functools.lru_cache(maxsize=4096)
def _experts_bytes(device_index: int, rows: int, experts: int) -> int:
    n = _wsm.lib().wsm_expert_gemm_workspace_bytes(rows, experts)
    if n == 0:
        raise _wsm.WsmError(_wsm.WSM_ERR_UNSUPPORTED, "wsm_expert_gemm_workspace_bytes", _wsm.last_error())
    return n


def _pack_cache(k_cache, v_cache, k_scale, v_scale, device):
    pages, page, heads, dim = shape = _tensor("k_cache", k_cache, 4, device)
    if _tensor("v_cache", v_cache, 4, device, k_cache.dtype) != shape:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} differ in shape")
    code = _dtype("k_cache", k_cache, (_BF16, _FP16, _E4M3))
    ks, vs = k_cache.stride(), v_cache.stride()
    return shape, code, _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
                                    pages, page, heads, dim, code, k_scale, v_scale)


@_on_stream
def paged_cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       slots: torch.Tensor, *, k_scale: float = 1.0, v_scale: float = 1.0) -> None:
    """Write new tokens' keys and values into their slots of a paged cache.

    k, v: [tokens, kv_heads, head_dim] bf16 or fp16, any strides that are
    multiples of 16 bytes (slices of a fused qkv projection).  k_cache,
    v_cache: [pages, page_size, kv_heads, head_dim], of the same type or
    float8_e4m3fn (then value / scale is stored), in any order of the first
    three dimensions.  slots: [tokens] int64, page * page_size + place in the
    page; negative: the row is skipped.  Slots of one call must differ.
    """
    device = k.device if isinstance(k, torch.Tensor) else None
    tokens, heads, dim = shape = _tensor("k", k, 3)
    if _tensor("v", v, 3, device, k.dtype) != shape:
        raise ValueError(f"k {tuple(shape)} and v {tuple(v.shape)} differ in shape")
    cache_shape, _, cache = _pack_cache(k_cache, v_cache, k_scale, v_scale, device)
    if cache_shape[2:] != shape[1:]:
        raise ValueError(f"k {tuple(shape)} does not fit a cache of {tuple(cache_shape)}")
    if _tensor("slots", slots, 1, device, torch.int64) != (tokens,):
        raise ValueError(f"slots must be [{tokens}]")
    ks, vs = k.stride(), v.stride()
    rows = _ROWS.pack(k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1], slots.data_ptr(), tokens,
                      _dtype("k", k, (_BF16, _FP16)))
    _wsm._check(_wsm.lib().wsm_paged_cache_append(cache, rows, _current(device)), "wsm_paged_cache_append")


@_on_stream
def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    lengths: torch.Tensor, out: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                    window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0,
                    lse: Optional[torch.Tensor] = None) -> torch.Tensor:
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
    batch, heads, dim = shape = _tensor("q", q, 3)
    device = q.device
    code = _dtype("q", q, (_BF16, _FP16))
    cache_shape, cache_code, cache = _pack_cache(k_cache, v_cache, k_scale, v_scale, device)
    if cache_shape[3] != dim:
        raise ValueError(f"q {tuple(shape)} does not fit a cache of {tuple(cache_shape)}")
    if cache_code != _E4M3 and cache_code != code:
        raise TypeError(f"q is {q.dtype}, the cache {k_cache.dtype}")
    table_shape = _tensor("block_table", block_table, 2, device, torch.int32)
    if table_shape[0] != batch:
        raise ValueError(f"block_table must have {batch} rows")
    if _tensor("lengths", lengths, 1, device, torch.int32) != (batch,):
        raise ValueError(f"lengths must be [{batch}]")
    if out is None:
        out = q.new_empty(shape)
    elif _tensor("out", out, 3, device, q.dtype) != shape:
        raise ValueError(f"out must be {list(shape)}")
    if lse is not None:
        _output("lse", lse, (batch, heads), device, torch.float32)
    if batch == 0:
        return out
    n = _attention_bytes(device.index, batch, dim)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    qs, os_ = q.stride(), out.stride()
    args = _ATTENTION.pack(q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else 0,
                           block_table.data_ptr(), lengths.data_ptr(), qs[0], qs[1], os_[0], os_[1],
                           block_table.stride(0), ws.data_ptr(), n, batch, heads, table_shape[1], window, code,
                           dim ** -0.5 if scale is None else scale)
    _wsm._check(_wsm.lib().wsm_paged_attention(cache, args, _current(device)), "wsm_paged_attention")
    return out


@_on_stream
def expert_gemm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                epilogue: int = 0, row_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Products grouped by expert: y[r] = x[r] @ w[e].T for the rows
    offsets[e] <= r < offsets[e + 1] of expert e; returns y.

    x: [rows, K], w: [experts, N, K], both bf16 or both fp16; offsets:
    [experts + 1] int32 on the device.  With epilogue=EPI_SILU_MUL, w holds
    gate and up rows in alternating blocks of 8 and y is [rows, N / 2] =
    silu(gate) * up.  row_scale: [rows] fp32 factors of the results (router
    weights).  Rows outside all experts are left as they were: in a new y
    they are undefined.
    """
    rows, k = _tensor("x", x, 2)
    device = x.device
    code = _dtype("x", x, (_BF16, _FP16))
    experts, n, wk = _tensor("w", w, 3, device, x.dtype)
    if wk != k:
        raise ValueError(f"shapes x{tuple(x.shape)} w{tuple(w.shape)} do not form x[rows, K] . w[e][N, K]^T")
    if _tensor("offsets", offsets, 1, device, torch.int32) != (experts + 1,):
        raise ValueError(f"offsets must be [{experts + 1}]")
    shape = (rows, n // 2 if epilogue == _wsm.EPI_SILU_MUL else n)
    if y is None:
        y = x.new_empty(shape)
    elif _tensor("y", y, 2, device, x.dtype) != shape:
        raise ValueError(f"y must be {list(shape)}")
    if row_scale is not None and _tensor("row_scale", row_scale, 1, device, torch.float32) != (rows,):
        raise ValueError(f"row_scale must be [{rows}]")
    nbytes = _experts_bytes(device.index, rows, experts)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    we, wr, _ = w.stride()
    args = _EXPERTS.pack(x.data_ptr(), w.data_ptr(), y.data_ptr(), offsets.data_ptr(),
                         row_scale.data_ptr() if row_scale is not None else 0, x.stride(0), we, wr, y.stride(0),
                         ws.data_ptr(), nbytes, rows, experts, n, k, epilogue, code)
    _wsm._check(_wsm.lib().wsm_expert_gemm(args, _current(device)), "wsm_expert_gemm")
    return y


@_on_stream
def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, top: int = 0) -> TokenLogprobs:
    """Log probabilities of given tokens, the entropy of each row's
    distribution and its `top` (at most 32) likeliest tokens.

    logits: [rows, vocab] fp32 (skinny_gemm's yf32), bf16 or fp16, rows any
    distance apart.  tokens: [rows] int64; a negative one asks for nothing and
    gets 0, as does every row without tokens.  Alternatives come likeliest
    first, equal ones by the lower index; places that no token with a
    probability above 0 takes hold -1 and -infinity.
    """
    rows, vocab = _tensor("logits", logits, 2)
    device = logits.device
    code = _dtype("logits", logits, (_FP32, _BF16, _FP16))
    if tokens is not None and _tensor("tokens", tokens, 1, device, torch.int64) != (rows,):
        raise ValueError(f"tokens must be [{rows}]")
    both = torch.empty((2, rows), dtype=torch.float32, device=device)
    logprob, entropy = both[0], both[1]
    top_lp = torch.empty((rows, max(top, 0)), dtype=torch.float32, device=device)
    top_ids = torch.empty((rows, max(top, 0)), dtype=torch.int64, device=device)
    at = both.data_ptr()
    args = _LOGPROBS.pack(logits.data_ptr(), tokens.data_ptr() if tokens is not None else 0, at, at + 4 * rows,
                          top_ids.data_ptr(), top_lp.data_ptr(), logits.stride(0), rows, vocab, top, code)
    _wsm._check(_wsm.lib().wsm_token_logprobs(args, _current(device)), "wsm_token_logprobs")
    return TokenLogprobs(logprob, entropy, top_ids, top_lp)


def operator_status(stream=None) -> int:
    """Synchronise the stream; 0, or the first error that a decode-step
    operator recorded on the current device, on any stream, since the last
    check: WSM_ERR_INVALID for an index out of range (last_error() says
    which), WSM_ERR_TIMEOUT for a device-side wait that ran out."""
    code = ctypes.c_int(0)
    rc = _wsm.lib().wsm_operator_status(_wsm._stream_handle(stream), ctypes.byref(code))
    if rc not in (_wsm.WSM_OK, _wsm.WSM_ERR_INVALID, _wsm.WSM_ERR_TIMEOUT):
        raise _wsm.WsmError(rc, "wsm_operator_status", _wsm.last_error())
    return code.value
