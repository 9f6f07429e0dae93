"""Plain reference of the 8-bit cache and of the rotating appends, in numpy: e4m3 by its value table, the append
token by token in float32 steps (the arithmetic the kernels promise bit for bit), attention in float64."""
from __future__ import annotations

import numpy as np


def _table():
    v = np.empty(256, np.float64)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = np.nan if (b & 0x7F) == 0x7F else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[b] = -x if s else x
    return v


E4M3 = _table()
_POS = E4M3[:0x7F]  # the 127 non-negative finite values, increasing with their byte


def e4m3_bytes(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 bytes of x (float64 or float32), ties to the even mantissa, saturating; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    up, down = _POS[hi] - a, a - _POS[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    out = (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), out)


def same_bytes(a: np.ndarray, b: np.ndarray) -> bool:
    """Equal bytes, any NaN pattern standing for any other."""
    nan = ((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)
    return bool(np.all((a == b) | nan))


def pow2_scale(amax: float) -> np.float32:
    e = -64
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def rotate(x: np.ndarray, cos_sin: np.ndarray, positions: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [T, H, d] turned, in x's own precision: every product and sum rounded once."""
    r = cos_sin.shape[1]
    c = cos_sin[positions][:, None, :r // 2].astype(x.dtype)
    s = cos_sin[positions][:, None, r // 2:].astype(x.dtype)
    y = x.copy()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    with np.errstate(invalid="ignore", over="ignore"):
        p, q = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = p, q
    else:
        y[..., :r // 2], y[..., r // 2:r] = p, q
    return y


def append_rows(x: np.ndarray, cache: np.ndarray, scale: np.ndarray, slots: np.ndarray) -> None:
    """Append float32 rows x [T, H, d] to e4m3 bytes cache [NB, H, bs, d] with scale [NB, H], in place."""
    nb, H, bs, _ = cache.shape
    written = [t for t in range(len(slots)) if 0 <= slots[t] < nb * bs]
    runs = []
    for t in written:
        if not runs or slots[runs[-1][0]] // bs != slots[t] // bs:
            runs.append([])
        runs[-1].append(t)
    for run in runs:
        blk, rows = slots[run[0]] // bs, slots[run] % bs
        for h in range(H):
            m = np.abs(x[run, h])
            want = pow2_scale(float(np.max(m[np.isfinite(m)], initial=0.0)))
            if 0 in rows:
                new = want
            else:
                new = np.maximum(scale[blk, h], want)
                if new > scale[blk, h]:
                    ratio = np.float32(scale[blk, h]) / new
                    cache[blk, h] = e4m3_bytes(E4M3[cache[blk, h]].astype(np.float32) * ratio)
            with np.errstate(invalid="ignore"):
                cache[blk, h, rows] = e4m3_bytes(x[run, h] / new)
            scale[blk, h] = new


def quantise_pool(x: np.ndarray):
    """Bytes and scales of a whole pool x [NB, H, bs, d] of float32 rows."""
    scale = np.vectorize(pow2_scale, otypes=[np.float32])(np.abs(x).max((2, 3)))
    return e4m3_bytes(x / scale[:, :, None, None]), scale


def values(cache: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """What the bytes stand for, float64."""
    return E4M3[cache] * scale.astype(np.float64)[:, :, None, None]


def attention(q, k_pool, v_pool, tables, ctx, scale, new=None, bounds=False):
    """Attention in float64 of q [N, Hq, d] over pools [NB, H, bs, d] (float64): sequence s brings its last new[s]
    (default 1) tokens, causal.  Sequences without context give zeros.  With ``bounds`` also, per output element,
    sum_j w_j |v_j|, and per (token, head) the largest sum_i |scale q_i k_ji| over its keys."""
    q = np.asarray(q, np.float64)
    hkv, bs, d = k_pool.shape[1:]
    group = q.shape[1] // hkv
    out, mean_abs, dots = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
    new = np.ones(len(ctx), int) if new is None else np.asarray(new)
    at = 0
    for s, L in enumerate(ctx):
        n = int(new[s])
        L = int(L)
        if L and n:
            ids = tables[s, :-(-L // bs)]
            k = k_pool[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :L]
            v = v_pool[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :L]
            seen = np.arange(L)[None, None] <= np.arange(L - n, L)[None, :, None]
            for h in range(hkv):
                heads = slice(h * group, (h + 1) * group)
                qh = q[at:at + n, heads].transpose(1, 0, 2)
                z = np.where(seen, np.matmul(qh, k[h].T) * scale, -np.inf)
                w = np.exp(z - z.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                out[at:at + n, heads] = np.matmul(w, v[h]).transpose(1, 0, 2)
                if bounds:
                    mean_abs[at:at + n, heads] = np.matmul(w, np.abs(v[h])).transpose(1, 0, 2)
                    b = np.where(seen, np.matmul(np.abs(qh), np.abs(k[h]).T) * abs(scale), 0.0)
                    dots[at:at + n, heads] = b.max(-1).T
        at += n
    return (out, mean_abs, dots) if bounds else out
