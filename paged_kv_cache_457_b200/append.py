"""Appends of a step's keys and values to the paged caches beyond the plain 16-bit copy of
:func:`write_kv`: with the rotary position embedding applied on the way, and into caches held in
8 bits (e4m3) with one scale for each block and kv head.

Argument marshalling only; the work is one launch of the library's CUDA kernels per call (two for long inputs into 8 bits).
8-bit caches are ``torch.float8_e4m3fn`` tensors ``[num_blocks, num_kv_heads, block_size, head_dim]``
with float32 scales ``[num_blocks, num_kv_heads]``: a stored value stands for value * scale.

A decode step's calls last a few microseconds on the GPU, so the checks here look at each property of
a tensor once and build their messages only when one fails.
"""
from __future__ import annotations

import ctypes
import sys

import torch

from . import PagedAttentionError, _DTYPES, _cache_geometry, _check, _need_cuda, load_library

_package = sys.modules[__package__]

F8 = torch.float8_e4m3fn
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


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


def library() -> ctypes.CDLL:
    """The loaded library (loading it takes a lock, which a call need not)."""
    return _package._lib or load_library()


def stream_of(dev: torch.device) -> int:
    """The current stream of ``dev`` as the C ABI takes it."""
    if _raw_stream is None or dev.index is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream(dev.index)


def on_device(dev: torch.device, f, *args) -> int:
    """f(*args) with ``dev`` the current device: the library launches on the current one."""
    if dev.index == torch.cuda.current_device():
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def need_cuda(**tensors) -> None:
    """Refuses whatever is not a CUDA tensor on the device of the first one (None: an argument left out)."""
    dev = None
    for name, t in tensors.items():
        if t is not None:
            _need_cuda(name, t, dev)
            dev = dev or t.device


def same_device(k_cache, *tensors) -> torch.device | None:
    """The CUDA device all of these tensors lie on, None if they do not (:func:`need_cuda` then says which)."""
    try:
        dev = k_cache.device
        if dev.type != "cuda":
            return None
        for t in tensors:
            if t is not None and t.device != dev:
                return None
        return dev
    except AttributeError:
        return None


def fp8_geometry(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
    """Sizes (num_blocks, num_kv_heads, block_size, head_dim) of a checked 8-bit cache."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise PagedAttentionError("k_cache/v_cache must both be [num_blocks, num_kv_heads, block_size, head_dim]")
    if k_cache.dtype is not F8 or v_cache.dtype is not F8:
        raise PagedAttentionError("8-bit caches must be float8_e4m3fn")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise PagedAttentionError("caches must be contiguous")
    heads = shape[:2]
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dtype is not torch.float32 or t.shape != heads or not t.is_contiguous():
            raise PagedAttentionError(f"{name} must be a contiguous float32 [num_blocks, num_kv_heads] tensor")
    return shape


def token_stride(name: str, t: torch.Tensor, T: int, H: int, d: int, dtype) -> int:
    """Checks rows [T, H, d] (heads and dims contiguous within a token) and returns their token stride."""
    if t.dtype is not dtype or t.shape != (T, H, d):
        raise PagedAttentionError(f"{name} must be {[T, H, d]} of {dtype}, not {list(t.shape)} of {t.dtype}")
    if T == 0:
        return H * d
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and H > 1):
        raise PagedAttentionError(f"{name}: heads and dims must be contiguous within a token")
    return s0 if T > 1 else H * d


def _tokens(slot_mapping: torch.Tensor) -> int:
    shape = slot_mapping.shape
    if slot_mapping.dtype is not torch.int64 or len(shape) != 1 or not slot_mapping.is_contiguous():
        raise PagedAttentionError("slot_mapping must be a contiguous int64 [T] tensor")
    return shape[0]


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """Angles for the rotating appends: float32 [max_positions, rot_dim], row p holding
    cos(p * base^(-2i / rot_dim)) for i < rot_dim / 2 and then the sines.  Computed in 64 bits: at far
    positions a 32-bit product p * frequency has lost the angle's fraction."""
    inv = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _rope_args(q, q_out, T, d, dtype, positions, cos_sin, dev):
    """Checked (q pointer, q_out, its pointer, num_q_heads, q stride, q_out stride, rot_dim, max_positions)."""
    if positions.dtype is not torch.int64 or positions.shape != (T,) or not positions.is_contiguous():
        raise PagedAttentionError("positions must be a contiguous int64 [T] tensor")
    angles = cos_sin.shape
    if cos_sin.dtype is not torch.float32 or len(angles) != 2 or not cos_sin.is_contiguous():
        raise PagedAttentionError("cos_sin must be a contiguous float32 [max_positions, rot_dim] tensor")
    max_positions, rot = angles
    if q is None:
        if q_out is not None:
            raise PagedAttentionError("q_out without q")
        return None, None, None, 0, 0, 0, rot, max_positions
    shape = q.shape
    if len(shape) != 3 or shape[1] == 0:
        raise PagedAttentionError("q must be [T, Hq, d]")
    hq = shape[1]
    qs = token_stride("q", q, T, hq, d, dtype)
    if q_out is None:
        q_out = torch.empty((T, hq, d), dtype=dtype, device=dev)
        qos = hq * d
    else:
        qos = token_stride("q_out", q_out, T, hq, d, dtype)
    return q.data_ptr(), q_out, q_out.data_ptr(), hq, qs, qos, rot, max_positions


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
    dev = same_device(k_cache, k, v, v_cache, slot_mapping, positions, cos_sin, q, q_out)
    if dev is None:
        need_cuda(k_cache=k_cache, k=k, v=v, v_cache=v_cache, slot_mapping=slot_mapping,
                  positions=positions, cos_sin=cos_sin, q=q, q_out=q_out)
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape or dtype not in _DTYPES or v_cache.dtype is not dtype \
            or not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        _cache_geometry(k_cache, v_cache)  # says what is wrong
    nb, hkv, bs, d = shape
    T = _tokens(slot_mapping)
    ks, vs = token_stride("k", k, T, hkv, d, dtype), token_stride("v", v, T, hkv, d, dtype)
    qp, q_out, qop, hq, qs, qos, rot, maxp = _rope_args(q, q_out, T, d, dtype, positions, cos_sin, dev)
    rc = on_device(dev, library().pa_rope_write_kv, qp, k.data_ptr(), v.data_ptr(), qop, k_cache.data_ptr(),
                   v_cache.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), T, hq, hkv, d,
                   rot, 1 if interleaved else 0, bs, nb, maxp, qs, ks, vs, qos, _DTYPES[dtype], stream_of(dev))
    if rc:
        _check(rc, "pa_rope_write_kv")
    return q_out


def write_kv_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 k_scale: torch.Tensor, v_scale: torch.Tensor, slot_mapping: torch.Tensor) -> None:
    """Quantise k[t], v[t] ([T, Hkv, d], float16 or bfloat16) into slot_mapping[t] of 8-bit caches, in place.

    A (block, head)'s scale is the smallest power of two that holds its rows' magnitudes (at most 448 scales):
    it starts anew when row 0 of the block is written and grows, with the block's bytes re-scaled, when a later
    row needs it.  The tokens of one block must stand together in ``slot_mapping`` (skipped ones may lie between).
    """
    dev = same_device(k_cache, k, v, v_cache, k_scale, v_scale, slot_mapping)
    if dev is None:
        need_cuda(k_cache=k_cache, k=k, v=v, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                  slot_mapping=slot_mapping)
    nb, hkv, bs, d = fp8_geometry(k_cache, v_cache, k_scale, v_scale)
    dtype = k.dtype
    if dtype not in _DTYPES:
        raise PagedAttentionError("k and v must be float16 or bfloat16")
    T = _tokens(slot_mapping)
    ks, vs = token_stride("k", k, T, hkv, d, dtype), token_stride("v", v, T, hkv, d, dtype)
    rc = on_device(dev, library().pa_write_kv_fp8, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
                   v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), slot_mapping.data_ptr(), T, hkv, d, bs,
                   nb, ks, vs, _DTYPES[dtype], stream_of(dev))
    if rc:
        _check(rc, "pa_write_kv_fp8")


def rope_write_kv_fp8(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                      slot_mapping: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                      interleaved: bool = False, q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """:func:`rope_write_kv` into 8-bit caches (scales as :func:`write_kv_fp8` keeps them); k is quantised from its
    fp32 rotation, the returned q has the type of q."""
    dev = same_device(k_cache, k, v, v_cache, k_scale, v_scale, slot_mapping, positions, cos_sin, q, q_out)
    if dev is None:
        need_cuda(k_cache=k_cache, k=k, v=v, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                  slot_mapping=slot_mapping, positions=positions, cos_sin=cos_sin, q=q, q_out=q_out)
    nb, hkv, bs, d = fp8_geometry(k_cache, v_cache, k_scale, v_scale)
    dtype = k.dtype
    if dtype not in _DTYPES:
        raise PagedAttentionError("k and v must be float16 or bfloat16")
    T = _tokens(slot_mapping)
    ks, vs = token_stride("k", k, T, hkv, d, dtype), token_stride("v", v, T, hkv, d, dtype)
    qp, q_out, qop, hq, qs, qos, rot, maxp = _rope_args(q, q_out, T, d, dtype, positions, cos_sin, dev)
    rc = on_device(dev, library().pa_rope_write_kv_fp8, qp, k.data_ptr(), v.data_ptr(), qop, k_cache.data_ptr(),
                   v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), slot_mapping.data_ptr(),
                   positions.data_ptr(), cos_sin.data_ptr(), T, hq, hkv, d, rot, 1 if interleaved else 0, bs, nb, maxp,
                   qs, ks, vs, qos, _DTYPES[dtype], stream_of(dev))
    if rc:
        _check(rc, "pa_rope_write_kv_fp8")
    return q_out
