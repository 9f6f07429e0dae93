"""Appends of a step's keys and values to the paged caches beyond the plain 16-bit copy of
:func:`write_kv`: with the rotary position embedding applied on the way, and into caches held in
8 bits (e4m3) with one scale for each block and kv head.

Argument marshalling only; the work is one launch of the library's CUDA kernels per call.
8-bit caches are ``torch.float8_e4m3fn`` tensors ``[num_blocks, num_kv_heads, block_size, head_dim]``
with float32 scales ``[num_blocks, num_kv_heads]``: a stored value stands for value * scale.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

F8 = torch.float8_e4m3fn


def bind(lib: ctypes.CDLL) -> None:
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "pa_rope_write_kv": [vp] * 9 + [i64] + [i32] * 6 + [i64] * 6 + [i32, vp],
        "pa_write_kv_fp8": [vp] * 7 + [i64, i32, i32, i32, i64, i64, i64, i32, vp],
        "pa_rope_write_kv_fp8": [vp] * 11 + [i64] + [i32] * 6 + [i64] * 6 + [i32, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = args


def on_device(dev: torch.device):
    """Makes ``dev`` current for a call when it is not already: the library launches on the current device."""
    return contextlib.nullcontext() if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def fp8_geometry(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
    """Sizes (num_blocks, num_kv_heads, block_size, head_dim) of a checked 8-bit cache."""
    from . import PagedAttentionError
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise PagedAttentionError("k_cache/v_cache must both be [num_blocks, num_kv_heads, block_size, head_dim]")
    if k_cache.dtype != F8 or v_cache.dtype != F8:
        raise PagedAttentionError("8-bit caches must be float8_e4m3fn")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise PagedAttentionError("caches must be contiguous")
    shape = k_cache.shape[:2]
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
            raise PagedAttentionError(f"{name} must be a contiguous float32 [num_blocks, num_kv_heads] tensor")
    return tuple(k_cache.shape)


def token_stride(name: str, t: torch.Tensor, shape, dtype) -> int:
    """Checks rows [T, H, d] (heads and dims contiguous within a token) and returns their token stride."""
    from . import PagedAttentionError
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise PagedAttentionError(f"{name} must be {list(shape)} of {dtype}, not {list(t.shape)} of {t.dtype}")
    T, H, d = shape
    if T == 0:
        return H * d
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and H > 1):
        raise PagedAttentionError(f"{name}: heads and dims must be contiguous within a token")
    return s0 if T > 1 else H * d


def _slots(slot_mapping: torch.Tensor) -> int:
    from . import PagedAttentionError
    if slot_mapping.dtype != torch.int64 or slot_mapping.dim() != 1 or not slot_mapping.is_contiguous():
        raise PagedAttentionError("slot_mapping must be a contiguous int64 [T] tensor")
    return int(slot_mapping.shape[0])


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """Angles for the rotating appends: float32 [max_positions, rot_dim], row p holding
    cos(p * base^(-2i / rot_dim)) for i < rot_dim / 2 and then the sines.  Computed in 64 bits: at far
    positions a 32-bit product p * frequency has lost the angle's fraction."""
    inv = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _rope_args(q, q_out, T, d, dtype, positions, cos_sin, dev):
    """Checked (q_out, num_q_heads, q stride, q_out stride, rot_dim, max_positions)."""
    from . import PagedAttentionError, _need_cuda
    _need_cuda("positions", positions, dev)
    _need_cuda("cos_sin", cos_sin, dev)
    if positions.dtype != torch.int64 or tuple(positions.shape) != (T,) or not positions.is_contiguous():
        raise PagedAttentionError("positions must be a contiguous int64 [T] tensor")
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise PagedAttentionError("cos_sin must be a contiguous float32 [max_positions, rot_dim] tensor")
    max_positions, rot = cos_sin.shape
    if q is None:
        if q_out is not None:
            raise PagedAttentionError("q_out without q")
        return None, 0, 0, 0, rot, max_positions
    _need_cuda("q", q, dev)
    if q.dim() != 3 or q.shape[1] == 0:
        raise PagedAttentionError("q must be [T, Hq, d]")
    hq = q.shape[1]
    qs = token_stride("q", q, (T, hq, d), dtype)
    if q_out is None:
        q_out = torch.empty((T, hq, d), dtype=dtype, device=dev)
        return q_out, hq, qs, hq * d, rot, max_positions
    _need_cuda("q_out", q_out, dev)
    return q_out, hq, qs, token_stride("q_out", q_out, (T, hq, d), dtype), rot, max_positions


def rope_write_kv(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, slot_mapping: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                  interleaved: bool = False, q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Turn q ([T, Hq, d]) and k ([T, Hkv, d]) by their tokens' positions (int64 [T]) and store the turned k, and v,
    at slot_mapping[t] of the 16-bit caches, in place; returns the turned q.

    ``cos_sin``: float32 [max_positions, rot_dim] (:func:`rope_table`); the first rot_dim dims of a head are turned,
    in pairs (i, i + rot_dim / 2), or (2i, 2i + 1) when ``interleaved``.  ``q_out`` may be q itself (in place).
    A negative position marks padding: the token is left out altogether (its row of q_out is not written); a
    negative slot leaves out its K/V only.  ``q`` may be None.
    """
    from . import _DTYPES, _cache_geometry, _check, _need_cuda, _stream, load_library
    dev = k_cache.device
    for name, t in (("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("slot_mapping", slot_mapping)):
        _need_cuda(name, t, dev)
    nb, hkv, bs, d = _cache_geometry(k_cache, v_cache)
    dtype = k_cache.dtype
    T = _slots(slot_mapping)
    ks, vs = token_stride("k", k, (T, hkv, d), dtype), token_stride("v", v, (T, hkv, d), dtype)
    q_out, hq, qs, qos, rot, maxp = _rope_args(q, q_out, T, d, dtype, positions, cos_sin, dev)
    with on_device(dev):
        rc = load_library().pa_rope_write_kv(
            q.data_ptr() if hq else None, k.data_ptr(), v.data_ptr(), q_out.data_ptr() if hq else None,
            k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(),
            cos_sin.data_ptr(), T, hq, hkv, d, rot, 1 if interleaved else 0, bs, nb, maxp, qs, ks, vs, qos,
            _DTYPES[dtype], _stream(dev))
    _check(rc, "pa_rope_write_kv")
    return q_out


def write_kv_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 k_scale: torch.Tensor, v_scale: torch.Tensor, slot_mapping: torch.Tensor) -> None:
    """Quantise k[t], v[t] ([T, Hkv, d], float16 or bfloat16) into slot_mapping[t] of 8-bit caches, in place.

    A (block, head)'s scale is the smallest power of two that holds its rows' magnitudes (at most 448 scales):
    it starts anew when row 0 of the block is written and grows, with the block's bytes re-scaled, when a later
    row needs it.  The tokens of one block must stand together in ``slot_mapping`` (skipped ones may lie between).
    """
    from . import PagedAttentionError, _DTYPES, _check, _need_cuda, _stream, load_library
    dev = k_cache.device
    for name, t in (("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("k_scale", k_scale),
                    ("v_scale", v_scale), ("slot_mapping", slot_mapping)):
        _need_cuda(name, t, dev)
    nb, hkv, bs, d = fp8_geometry(k_cache, v_cache, k_scale, v_scale)
    dtype = k.dtype
    if dtype not in _DTYPES:
        raise PagedAttentionError("k and v must be float16 or bfloat16")
    T = _slots(slot_mapping)
    ks, vs = token_stride("k", k, (T, hkv, d), dtype), token_stride("v", v, (T, hkv, d), dtype)
    with on_device(dev):
        rc = load_library().pa_write_kv_fp8(
            k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), slot_mapping.data_ptr(), T, hkv, d, bs, nb, ks, vs, _DTYPES[dtype], _stream(dev))
    _check(rc, "pa_write_kv_fp8")


def rope_write_kv_fp8(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                      slot_mapping: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                      interleaved: bool = False, q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """:func:`rope_write_kv` into 8-bit caches (scales as :func:`write_kv_fp8` keeps them); k is quantised from its
    fp32 rotation, the returned q has the type of q."""
    from . import PagedAttentionError, _DTYPES, _check, _need_cuda, _stream, load_library
    dev = k_cache.device
    for name, t in (("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("k_scale", k_scale),
                    ("v_scale", v_scale), ("slot_mapping", slot_mapping)):
        _need_cuda(name, t, dev)
    nb, hkv, bs, d = fp8_geometry(k_cache, v_cache, k_scale, v_scale)
    dtype = k.dtype
    if dtype not in _DTYPES:
        raise PagedAttentionError("k and v must be float16 or bfloat16")
    T = _slots(slot_mapping)
    ks, vs = token_stride("k", k, (T, hkv, d), dtype), token_stride("v", v, (T, hkv, d), dtype)
    q_out, hq, qs, qos, rot, maxp = _rope_args(q, q_out, T, d, dtype, positions, cos_sin, dev)
    with on_device(dev):
        rc = load_library().pa_rope_write_kv_fp8(
            q.data_ptr() if hq else None, k.data_ptr(), v.data_ptr(), q_out.data_ptr() if hq else None,
            k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            slot_mapping.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), T, hq, hkv, d, rot,
            1 if interleaved else 0, bs, nb, maxp, qs, ks, vs, qos, _DTYPES[dtype], _stream(dev))
    _check(rc, "pa_rope_write_kv_fp8")
    return q_out
