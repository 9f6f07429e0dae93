"""Attention over paged caches held in 8 bits (e4m3) with one scale for each block and kv head.

Argument marshalling only; caches and scales as :mod:`.append` describes and fills them.
"""
from __future__ import annotations

import ctypes

import torch

from . import PagedAttentionError, _DTYPES, _check, _mapping, _need_cuda, _workspace, _workspace_use
from .append import fp8_geometry, library, need_cuda, on_device, same_device, stream_of, token_stride

PA_ERR_WORKSPACE = -7

# Kept apart from the 16-bit calls' workspaces: a captured graph of those goes on using the one kept for its stream, which
# a call here that needs more would free.
_workspaces: dict = {}


def bind(lib: ctypes.CDLL) -> None:
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sig = {
        "pa_decode_fp8_workspace_size": (sz, [i32] * 7),
        "pa_decode_fp8": (ctypes.c_int, [vp] * 7 + [f32, vp] + [i32] * 5 + [i64, i32, i32, i64, i64, i32, i32, vp, sz,
                                                                            vp]),
        "pa_prefill_fp8_workspace_size": (sz, [i32, i64, i32, i32, i32, i32, i32]),
        "pa_prefill_fp8": (ctypes.c_int, [vp] * 8 + [f32, vp, i32, i64] + [i32] * 4 + [i64, i32, i32, i64, i64, i32, vp,
                                                                                     sz, vp]),
        "pa_copy_blocks_fp8": (ctypes.c_int, [vp] * 5 + [i64, i32, i32, i32, i64, vp]),
        "pa_swap_blocks_fp8": (ctypes.c_int, [vp] * 9 + [i64, i32, i32, i32, i64, i64, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args


def _tables(block_tables: torch.Tensor, context_lens: torch.Tensor, S: int) -> int:
    """Checks the batch's tables and lengths; returns the table's row stride."""
    shape = block_tables.shape
    if block_tables.dtype is not torch.int32 or len(shape) != 2 or shape[0] != S:
        raise PagedAttentionError("block_tables must be int32 [S, max_blocks] with contiguous rows")
    s0, s1 = block_tables.stride()
    if s1 != 1 and shape[1] > 1:
        raise PagedAttentionError("block_tables must be int32 [S, max_blocks] with contiguous rows")
    if context_lens.dtype is not torch.int32 or context_lens.shape != (S,) or not context_lens.is_contiguous():
        raise PagedAttentionError("context_lens must be a contiguous int32 [S] tensor")
    if S > 1 and s0 < shape[1]:
        raise PagedAttentionError("rows of block_tables must not overlap")
    return s0 if S > 1 else max(1, shape[1])


def _run(dev, what, size, sizes, call, args, workspace):
    """call(*args, workspace pointer, bytes, stream) with the caller's workspace, or with one kept per device and stream
    (of size(*sizes) bytes), on which one call at a time enqueues its operations.  A capture gets its own, from the
    graph's pool: a captured graph may be replayed beside other calls and must neither share theirs nor outlive it."""
    stream = stream_of(dev)
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise PagedAttentionError("workspace must be a contiguous tensor on the caches' device")
        rc = call(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream)
    elif torch.cuda.is_current_stream_capturing():
        n = int(size(*sizes))
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        rc = call(*args, ws.data_ptr() if n else None, n, stream)
    else:
        with _workspace_use:
            ws = _workspaces.get((dev.index, stream))
            rc = call(*args, ws.data_ptr(), ws.numel(), stream) if ws is not None else call(*args, None, 0, stream)
            if rc == PA_ERR_WORKSPACE:
                ws = _workspace(dev, stream, int(size(*sizes)), _workspaces)
                rc = call(*args, ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0, stream)
    if rc:
        _check(rc, what)


def decode_fp8_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len,
                              partition_tokens: int = 0) -> int:
    """Device workspace bytes of :func:`decode_fp8` for these sizes on the current device (0: none, or bad input)."""
    return int(library().pa_decode_fp8_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                           max_context_len, partition_tokens))


def decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
               max_context_len: int | None = None, out: torch.Tensor | None = None, partition_tokens: int = 0,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """:func:`decode` over an 8-bit cache: attention of q ([S, Hq, d], float16 or bfloat16) over each sequence's
    context; returns out ([S, Hq, d], q's dtype).  Other arguments as :func:`decode`; ``partition_tokens`` is rounded
    up to a multiple of 32, and to 64 at least."""
    dev = same_device(k_cache, q, v_cache, k_scale, v_scale, block_tables, context_lens)
    if dev is None:
        need_cuda(k_cache=k_cache, q=q, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                  block_tables=block_tables, context_lens=context_lens)
    nb, hkv, bs, d = fp8_geometry(k_cache, v_cache, k_scale, v_scale)
    dtype, shape = q.dtype, q.shape
    if dtype not in _DTYPES or len(shape) != 3:
        raise PagedAttentionError("q must be float16 or bfloat16 [S, Hq, d]")
    S, hq = shape[0], shape[1]
    qs = token_stride("q", q, S, hq, d, dtype)
    ts = _tables(block_tables, context_lens, S)
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty((S, hq, d), dtype=dtype, device=dev)
        os_ = hq * d
    else:
        _need_cuda("out", out, dev)
        os_ = token_stride("out", out, S, hq, d, dtype)
    if max_context_len is None:
        max_context_len = context_lens.max().item() if S else 0
    max_context_len, partition_tokens, scale = int(max_context_len), int(partition_tokens), float(scale)
    lib = library()

    on_device(dev, _run, dev, "pa_decode_fp8", lib.pa_decode_fp8_workspace_size,
              (S, hq, hkv, d, bs, max_context_len, partition_tokens), lib.pa_decode_fp8,
              (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
               block_tables.data_ptr(), context_lens.data_ptr(), scale, out.data_ptr(), S, hq, hkv, d, bs, nb, ts,
               max_context_len, qs, os_, partition_tokens, _DTYPES[dtype]), workspace)
    return out


def prefill_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                v_scale: torch.Tensor, block_tables: torch.Tensor, query_start: torch.Tensor,
                context_lens: torch.Tensor, scale: float, max_query_len: int, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """:func:`prefill` over an 8-bit cache: causal attention of each sequence's new tokens (their K/V already written)
    over its context.  q: [N, Hq, d], float16 or bfloat16; other arguments as :func:`prefill`."""
    dev = same_device(k_cache, q, v_cache, k_scale, v_scale, block_tables, query_start, context_lens)
    if dev is None:
        need_cuda(k_cache=k_cache, q=q, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                  block_tables=block_tables, query_start=query_start, context_lens=context_lens)
    nb, hkv, bs, d = fp8_geometry(k_cache, v_cache, k_scale, v_scale)
    dtype, shape = q.dtype, q.shape
    if dtype not in _DTYPES or len(shape) != 3:
        raise PagedAttentionError("q must be float16 or bfloat16 [N, Hq, d]")
    N, hq = shape[0], shape[1]
    S = context_lens.shape[0]
    qs = token_stride("q", q, N, hq, d, dtype)
    ts = _tables(block_tables, context_lens, S)
    if query_start.dtype is not torch.int32 or query_start.shape != (S + 1,) or not query_start.is_contiguous():
        raise PagedAttentionError("query_start must be a contiguous int32 [S + 1] tensor")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty((N, hq, d), dtype=dtype, device=dev)
        os_ = hq * d
    else:
        _need_cuda("out", out, dev)
        os_ = token_stride("out", out, N, hq, d, dtype)
    max_query_len, scale = int(max_query_len), float(scale)
    lib = library()

    on_device(dev, _run, dev, "pa_prefill_fp8", lib.pa_prefill_fp8_workspace_size,
              (S, N, hq, hkv, d, bs, max_query_len), lib.pa_prefill_fp8,
              (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
               block_tables.data_ptr(), query_start.data_ptr(), context_lens.data_ptr(), scale, out.data_ptr(), S, N, hq,
               hkv, d, bs, nb, ts, max_query_len, qs, os_, _DTYPES[dtype]), workspace)
    return out


def copy_blocks_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                    block_mapping: torch.Tensor) -> None:
    """:func:`copy_blocks` for 8-bit caches: a block's bytes and the scales of its heads (copy-on-write)."""
    need_cuda(k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
    dev = k_cache.device
    nb, hkv, bs, d = fp8_geometry(k_cache, v_cache, k_scale, v_scale)
    m = _mapping(block_mapping, dev)
    rc = on_device(dev, library().pa_copy_blocks_fp8, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                   v_scale.data_ptr(), m.data_ptr(), m.shape[0], hkv, d, bs, nb, stream_of(dev))
    _check(rc, "pa_copy_blocks_fp8")


def swap_blocks_fp8(src_k: torch.Tensor, src_v: torch.Tensor, src_k_scale: torch.Tensor, src_v_scale: torch.Tensor,
                    dst_k: torch.Tensor, dst_v: torch.Tensor, dst_k_scale: torch.Tensor, dst_v_scale: torch.Tensor,
                    block_mapping: torch.Tensor, device: torch.device | None = None) -> None:
    """:func:`swap_blocks` for 8-bit pools with their scales; either pool may be pinned host memory."""
    pools = (src_k, src_v, src_k_scale, src_v_scale, dst_k, dst_v, dst_k_scale, dst_v_scale)
    for t in pools:
        if not (t.is_cuda or t.is_pinned()):
            raise PagedAttentionError("every pool and scale must be on the GPU or in pinned host memory")
    dev = device or next((t.device for t in pools if t.is_cuda), torch.device("cuda", torch.cuda.current_device()))
    snb, hkv, bs, d = fp8_geometry(src_k, src_v, src_k_scale, src_v_scale)
    dnb, *rest = fp8_geometry(dst_k, dst_v, dst_k_scale, dst_v_scale)
    if tuple(rest) != (hkv, bs, d):
        raise PagedAttentionError("pools must share heads, block size and head dim")
    m = _mapping(block_mapping, dev)
    rc = on_device(dev, library().pa_swap_blocks_fp8, *(t.data_ptr() for t in pools), m.data_ptr(), m.shape[0], hkv,
                   d, bs, snb, dnb, stream_of(dev))
    _check(rc, "pa_swap_blocks_fp8")
