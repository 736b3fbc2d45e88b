"""Binding of the paged key-value cache calls (w4a16_kv_append, w4a16_attention).

Argument checks and marshalling only, as in _lib. These calls sit in the inner
loop of a decode step, where a launch takes a few microseconds on the device:
the checks compare plain integers, and what depends on sizes alone (the
workspace's bytes) is computed once per size.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import W4A16_BF16, W4A16_F16, _check, _lib, _queue, _sz, _workspaces

_CODES = {torch.float16: W4A16_F16, torch.bfloat16: W4A16_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_capturing_here = torch.cuda.is_current_stream_capturing
_append_call = _lib.w4a16_kv_append
_attention_call = _lib.w4a16_attention


def _on_device(fn, device, *args, **kw):
    with torch.cuda.device(device):
        return fn(*args, **kw)


def _on_stream(fn, on, made, device, *args, **kw):
    """fn on stream `on`: the copies and the result (if `made` there) belong to it too."""
    if on.device != device:   # (the call would leave it for the caches' device)
        raise ValueError(f"the stream is one of {on.device}, the caches are on {device}")
    caller = torch.cuda.current_stream(on.device)
    with torch.cuda.stream(on):
        got = fn(*args, **kw)
    if made and got is not None:
        got.record_stream(caller)
    return got


def _rows(name, t, dtype, dev, dim):
    """t as [tokens][heads][dim] rows the kernels take: heads contiguous, the
    token stride a multiple of 8, the first on 16 bytes (a copy where they are
    not). Returns it with that stride and its shape."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor [tokens][heads][{dim}] on cuda:{dev}")
    s0, s1, s2 = t.stride()
    row = shape[1] * dim
    if shape[0] <= 1:
        s0 = row
    if s2 != 1 or s0 % 8 or s0 < row or (s1 != dim and shape[1] != 1) or t.data_ptr() % 16:
        return t.clone(memory_format=torch.contiguous_format), row, shape
    return t, s0, shape


def _out_rows(name, t, shape, dtype, dev):
    """The token stride of an output of token rows: its heads contiguous, any token stride."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} on cuda:{dev}")
    s0, s1, s2 = t.stride()
    row = shape[1] * shape[2]
    if shape[0] <= 1:
        s0 = row
    if s2 != 1 or s0 % 8 or s0 < row or (s1 != shape[2] and shape[1] != 1) or t.data_ptr() % 16:
        raise ValueError(f"{name}'s heads must be contiguous, its token stride a multiple of 8 and its start on 16 bytes")
    return s0


def _cache(k_cache, v_cache):
    """(type, its code, device, pages, kv_heads, page size, dim, page stride) of the two caches."""
    shape, dtype, dev = k_cache.shape, k_cache.dtype, k_cache.get_device()
    code = _CODES.get(dtype)
    if len(shape) != 4 or dev < 0 or code is None:
        raise ValueError("k_cache must be a float16 or bfloat16 CUDA tensor [pages][kv_heads][page_size][dim]")
    if v_cache.shape != shape or v_cache.dtype != dtype or v_cache.get_device() != dev:
        raise ValueError("v_cache must have k_cache's shape, type and device")
    pages, kvh, page, dim = shape
    s0, s1, s2, s3 = k_cache.stride()
    t0, t1, t2, t3 = v_cache.stride()
    row = page * dim
    # (a dimension of one may have any stride)
    if s2 != dim or t2 != dim or s3 != 1 or t3 != 1 or (kvh > 1 and (s1 != row or t1 != row)) or (pages > 1 and s0 != t0):
        raise ValueError("the caches' pages must be contiguous [kv_heads][page_size][dim], equally far apart")
    return dtype, code, dev, pages, kvh, page, dim, s0 if pages > 1 else kvh * row


def _index(name, t, dtype, shape, dev):
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{dev}")
    return t.data_ptr()


def kv_append(q, k, v, k_cache, v_cache, slots, positions=None, cos_sin=None, *, q_norm=None, k_norm=None, eps=1e-6,
              interleaved=False, q_out=None, stream=None):
    """New tokens' keys and values into a paged cache, with the heads' norms
    and the position rotation on the way (w4a16_kv_append).

    q [tokens][heads][dim] (None: keys and values alone), k and v
    [tokens][kv_heads][dim]: slices of a fused projection's output as they are.
    k_cache, v_cache [pages][kv_heads][page_size][dim]. slots int64 [tokens]:
    page * page_size + place, negative for a token that is not stored. positions
    int32 [tokens] and cos_sin float32 [max_positions][rot_dim] (cosines, then
    sines) rotate the first rot_dim values of q and k; q_norm and k_norm [dim]
    are the weights of a norm before it. Returns the queries, in q_out (which
    may be q) or a new tensor; a token whose slot or position is out of range is
    left out, and the next call reports it. Runs on `stream`, by default the current one."""
    if stream is not None:
        return _on_stream(kv_append, stream, q_out is None, k_cache.device, q, k, v, k_cache, v_cache, slots, positions, cos_sin,
                          q_norm=q_norm, k_norm=k_norm, eps=eps, interleaved=interleaved, q_out=q_out)
    dtype, code, dev, pages, kvh, page, dim, page_stride = _cache(k_cache, v_cache)
    if dev != _current_device():
        return _on_device(kv_append, dev, q, k, v, k_cache, v_cache, slots, positions, cos_sin, q_norm=q_norm,
                          k_norm=k_norm, eps=eps, interleaved=interleaved, q_out=q_out)
    k, ks, shape = _rows("k", k, dtype, dev, dim)
    v, vs, vshape = _rows("v", v, dtype, dev, dim)
    tokens = shape[0]
    if shape[1] != kvh or vshape != shape:
        raise ValueError(f"k and v must be [tokens][{kvh}][{dim}]")
    heads = qs = qos = 0
    q_ptr = qo_ptr = None
    if q is not None:
        in_place = q_out is q
        q, qs, qshape = _rows("q", q, dtype, dev, dim)
        heads = qshape[1]
        if qshape[0] != tokens:
            raise ValueError("q, k and v must have the same tokens")
        if q_out is None:
            q_out = torch.empty(qshape, dtype=dtype, device=k_cache.device)
            qos = heads * dim
        else:
            qos = _out_rows("q_out", q_out, qshape, dtype, dev)
            if in_place:
                qs = qos
        q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
    pos_ptr = cs_ptr = None
    rot = most = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2 or positions is None:
            raise ValueError("a rotation takes cos_sin [max_positions][rot_dim] and positions [tokens]")
        most, rot = cos_sin.shape
        cs_ptr = _index("cos_sin", cos_sin, torch.float32, (most, rot), dev)
        pos_ptr = _index("positions", positions, torch.int32, (tokens,), dev)
    status = _append_call(
        q_ptr, qs, k.data_ptr(), ks, v.data_ptr(), vs, code, tokens, heads, kvh, dim,
        _index("slots", slots, torch.int64, (tokens,), dev), pos_ptr, cs_ptr, most, rot, interleaved,
        None if q_norm is None else _index("q_norm", q_norm, dtype, (dim,), dev),
        None if k_norm is None else _index("k_norm", k_norm, dtype, (dim,), dev), eps, qo_ptr, qos,
        k_cache.data_ptr(), v_cache.data_ptr(), pages, page, page_stride, _raw_stream(dev))
    if status:
        _check("w4a16_kv_append", status)
    return q_out


@functools.lru_cache(maxsize=1024)
def attention_workspace_bytes(batch: int, heads: int, kv_heads: int, dim: int, max_q_len: int, max_kv_len: int,
                              window: int = 0, sinks: int = 0) -> int:
    b = _sz()
    _check("w4a16_attention_workspace_bytes", _lib.w4a16_attention_workspace_bytes(
        batch, heads, kv_heads, dim, max_q_len, max_kv_len, window, sinks, ctypes.byref(b)))
    return b.value


def attention(q, k_cache, v_cache, page_table, kv_lens, *, q_starts=None, max_q_len=None, max_kv_len=None, scale=None,
              window=0, sinks=0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of new tokens over a paged cache that already holds
    them (w4a16_attention).

    q [tokens][heads][dim]; k_cache, v_cache [pages][kv_heads][page_size][dim];
    page_table int32 [batch][columns]; kv_lens int32 [batch], each sequence's
    keys with its new ones. q_starts int32 [batch + 1]: sequence b's tokens are
    q_starts[b] .. q_starts[b + 1] - 1, at most max_q_len of them; without it
    each sequence has one. max_kv_len bounds kv_lens (by default what the page
    table can name); the tighter it is, the better the work is divided. scale:
    dim ** -0.5 by default. window and sinks: a token sees the last `window`
    keys (itself among them) and the first `sinks` of its sequence; 0: all.
    Returns the output, in `out` or a new tensor; lse float32 [tokens][heads],
    where given, gets ln sum exp of each row's scores. workspace: a Workspace
    instead of the stream's own (under capture, of memory of the graph).
    Rows of q that belong to no sequence are not written: a new tensor holds
    anything there. Single tokens over long caches belong in a call of their
    own, not beside prompts."""
    if stream is not None:
        return _on_stream(attention, stream, out is None, k_cache.device, q, k_cache, v_cache, page_table, kv_lens, q_starts=q_starts,
                          max_q_len=max_q_len, max_kv_len=max_kv_len, scale=scale, window=window, sinks=sinks, out=out,
                          lse=lse, workspace=workspace)
    dtype, code, dev, pages, kvh, page, dim, page_stride = _cache(k_cache, v_cache)
    if dev != _current_device():
        return _on_device(attention, dev, q, k_cache, v_cache, page_table, kv_lens, q_starts=q_starts,
                          max_q_len=max_q_len, max_kv_len=max_kv_len, scale=scale, window=window, sinks=sinks, out=out,
                          lse=lse, workspace=workspace)
    q, qs, shape = _rows("q", q, dtype, dev, dim)
    tokens, heads, _ = shape
    strides = page_table.stride()
    if len(strides) != 2 or page_table.dtype != torch.int32 or page_table.get_device() != dev:
        raise ValueError(f"page_table must be an int32 tensor [batch][pages of a sequence] on cuda:{dev}")
    batch, columns = page_table.shape
    if strides[1] != 1 and columns > 1:
        raise ValueError("page_table must be a tensor of contiguous rows")
    if max_kv_len is None:
        max_kv_len = columns * page
    elif max_kv_len > columns * page:
        raise ValueError(f"max_kv_len {max_kv_len} is more than the page table's {columns} pages of {page}")
    starts = None
    if q_starts is not None:
        if max_q_len is None:
            raise ValueError("q_starts needs max_q_len, the most tokens of a sequence")
        starts = _index("q_starts", q_starts, torch.int32, (batch + 1,), dev)
    else:
        if tokens != batch or max_q_len not in (None, 1):
            raise ValueError("without q_starts every sequence has one token")
        max_q_len = 1
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=k_cache.device)
        os = heads * dim
    else:
        os = _out_rows("out", out, shape, dtype, dev)
    nbytes = attention_workspace_bytes(batch, heads, kvh, dim, max_q_len, max_kv_len, window, sinks)
    raw = _raw_stream(dev)

    def call(ws, ws_len):
        return _attention_call(
            q.data_ptr(), qs, code, k_cache.data_ptr(), v_cache.data_ptr(), pages, page, page_stride, page_table.data_ptr(),
            strides[0] if batch > 1 else columns, _index("kv_lens", kv_lens, torch.int32, (batch,), dev), starts,
            tokens, batch, heads, kvh, dim, max_q_len, max_kv_len, dim ** -0.5 if scale is None else scale, window, sinks,
            out.data_ptr(), os, None if lse is None else _index("lse", lse, torch.float32, (tokens, heads), dev), ws,
            ws_len, raw)

    status = None
    if not nbytes:
        status = call(None, 0)
    elif workspace is None and not _capturing_here():
        ws = _workspaces.get((dev, raw))
        if ws is not None:
            with ws.lock:
                buf = ws.buf
                if buf is not None and buf.numel() >= nbytes and ws._alloc_stream.cuda_stream == raw:
                    status = call(buf.data_ptr(), nbytes)   # (allocated on this stream: nothing to record)
    if status is None:
        status = _queue(workspace, k_cache.device, torch.cuda.current_stream(dev), nbytes, call)
    if status:
        _check("w4a16_attention", status)
    return out
