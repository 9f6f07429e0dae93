"""Rotating appends into 16-bit caches and appends into 8-bit caches, against the plain reference.

The kernels promise the arithmetic of elementary float32 steps (products and sums rounded once each), so bytes,
scales and 16-bit rows are compared for equality with numpy's float32; the rotation is also held to the 64-bit
formula.  Tolerance there: three float32 roundings of values up to |a| + |b| (|cos|, |sin| <= 1, the table itself
is an input), 3 * 2^-24 (|a| + |b|), and half a step of the storage type (2^-11 or 2^-8 of the value, 2^-25 below
fp16's normal range)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref as R
import paged_kv_cache_457_b200 as pa
from gpu_util import TORCH_DT, require_gpu

pytestmark = pytest.mark.gpu

HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def rows(rng, dtype, *shape, gain=1.0):
    """Normal draws rounded to the storage type, as float32."""
    x = (rng.standard_normal(shape) * gain).astype(np.float32)
    return torch.from_numpy(x).to(TORCH_DT[dtype]).float().numpy()


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(TORCH_DT[dtype]) if dtype else t


def f8(b):
    return torch.from_numpy(np.ascontiguousarray(b)).cuda().view(torch.float8_e4m3fn)


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def round_to(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TORCH_DT[dtype]).float().numpy()


def token_mix(rng, nb, bs, singles, runs):
    """Slots of `singles` one-token appends and of runs (first row, tokens), each in blocks of its own."""
    free = list(rng.permutation(nb))
    out, pos = [], []
    for _ in range(singles):
        r = int(rng.integers(0, bs))
        out.append([free.pop() * bs + r])
        pos.append([int(rng.integers(0, 500))])
    for first, n in runs:
        blocks = [free.pop() for _ in range(-(-(first + n) // bs))]
        at = np.arange(first, first + n)
        out.append([int(blocks[i // bs] * bs + i % bs) for i in at])
        p0 = int(rng.integers(0, 500))
        pos.append(list(range(p0, p0 + n)))
    order = rng.permutation(len(out))
    return (np.array([s for i in order for s in out[i]], np.int64), np.array([p for i in order for p in pos[i]], np.int64))


SHAPES = [(8, 8, 64, 16, 64, False), (32, 8, 128, 16, 128, False), (12, 4, 128, 32, 128, True), (5, 5, 64, 32, 32, False),
          (16, 1, 128, 16, 16, False), (7, 1, 128, 32, 64, True), (3, 3, 64, 16, 16, True), (32, 4, 128, 16, 112, False)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs,rot,il", SHAPES)
def test_rope_write_kv(dtype, hq, hkv, d, bs, rot, il):
    require_gpu()
    rng = np.random.default_rng(d + rot + hq)
    nb, maxp = 64, 700
    slots, pos = token_mix(rng, nb, bs, 9, [(0, 1), (bs - 1, 2), (3, 2 * bs + 5), (0, bs)])
    T = len(slots)
    slots[4] = -1  # not stored, but its query is turned
    pos[7] = -1    # padding
    slots[9], pos[11] = nb * bs, maxp  # out of range: flagged
    qkv = rows(rng, dtype, T, hq + 2 * hkv, d, gain=2.0)
    cs = pa.rope_table(maxp, rot).numpy()
    kc0, vc0 = rows(rng, dtype, nb, hkv, bs, d), rows(rng, dtype, nb, hkv, bs, d)
    t = dev(qkv, dtype)
    q, k, v = t.split([hq, hkv, hkv], 1)
    kc, vc, q_out = dev(kc0, dtype), dev(vc0, dtype), torch.full((T, hq, d), 7.0, dtype=TORCH_DT[dtype], device="cuda")
    pa.device_status(clear=True)
    got = pa.rope_write_kv(q, k, v, kc, vc, dev(slots), dev(pos), dev(cs), interleaved=il, q_out=q_out)
    assert got is q_out
    assert pa.device_status() == pa.DEV_ERR_SLOT | pa.DEV_ERR_POSITION
    p = np.clip(pos, 0, maxp - 1)
    qt, kt = (R.rotate(x, cs, p, il) for x in (qkv[:, :hq], qkv[:, hq:hq + hkv]))
    want = round_to(qt, dtype)
    want[7], want[11] = 7.0, 0.0
    assert np.array_equal(q_out.float().cpu().numpy(), want)
    stored = [i for i in range(T) if i not in (4, 7, 9, 11)]
    for cache, c0, x in ((kc, kc0, round_to(kt, dtype)), (vc, vc0, qkv[:, hq + hkv:])):
        c0 = c0.copy()
        c0[slots[stored] // bs, :, slots[stored] % bs] = x[stored]
        assert np.array_equal(cache.float().cpu().numpy(), c0)
    # against the 64-bit formula
    keep = [i for i in range(T) if i not in (7, 11)]
    exact = R.rotate(qkv[keep, :hq].astype(np.float64), cs.astype(np.float64), p[keep], il)
    most = 2 * np.abs(qkv[keep, :hq]).max(-1, keepdims=True)  # at least |a| + |b| of every pair
    tol = 3 * 2.0 ** -24 * most + HALF_STEP[dtype] * (np.abs(exact) + 3 * 2.0 ** -24 * most) + 2.0 ** -25
    assert np.all(np.abs(q_out.float().cpu().numpy()[keep] - exact) <= tol)


def test_rope_in_place_without_q_and_other_stream():
    require_gpu()
    rng = np.random.default_rng(5)
    hq, hkv, d, bs, nb, T = 4, 2, 128, 16, 8, 20
    cs = pa.rope_table(64, d, device="cuda")
    q, k, v = (dev(rows(rng, "bf16", T, h, d), "bf16") for h in (hq, hkv, hkv))
    slots, pos = dev(np.arange(T) + 16), dev(np.arange(T))
    kc, vc = (torch.zeros((nb, hkv, bs, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ref = pa.rope_write_kv(q, k, v, kc, vc, slots, pos, cs)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q2 = q.clone()
        assert pa.rope_write_kv(q2, k, v, kc2, vc2, slots, pos, cs, q_out=q2) is q2
    side.synchronize()
    assert torch.equal(q2, ref) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    kc2.zero_(), vc2.zero_()
    assert pa.rope_write_kv(None, k, v, kc2, vc2, slots, pos, cs) is None
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    # no tokens: nothing happens
    empty = torch.empty((0,), dtype=torch.int64, device="cuda")
    n0 = pa.launch_count()
    assert pa.rope_write_kv(q[:0], k[:0], v[:0], kc2, vc2, empty, empty, cs).shape == (0, hq, d)
    assert pa.launch_count() == n0 and pa.device_status() == 0


def fp8_state(rng, nb, hkv, bs, d):
    kb, ks = R.quantise_pool(rng.standard_normal((nb, hkv, bs, d)).astype(np.float32))
    vb, vs = R.quantise_pool(rng.standard_normal((nb, hkv, bs, d)).astype(np.float32))
    return kb, ks, vb, vs


def check_fp8(kc, ks, vc, vs, want):
    for got, ref in ((ks, want[1]), (vs, want[3])):
        assert np.array_equal(got.cpu().numpy(), ref)
    for got, ref in ((kc, want[0]), (vc, want[2])):
        assert R.same_bytes(u8(got), ref)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("hq,hkv,d,bs,rot,il", SHAPES)
@pytest.mark.parametrize("gain", [0.01, 1.0, 300.0])
def test_append_fp8(dtype, rope, hq, hkv, d, bs, rot, il, gain):
    require_gpu()
    rng = np.random.default_rng(d + rot + hq)
    nb, maxp = 64, 700
    slots, pos = token_mix(rng, nb, bs, 9, [(0, 1), (bs - 1, 2), (3, 2 * bs + 5), (0, bs), (1, bs - 1)])
    T = len(slots)
    slots[4], slots[9] = -1, nb * bs
    if rope:
        pos[7], pos[11] = -1, maxp
    qkv = rows(rng, dtype, T, hq + 2 * hkv, d, gain=gain)
    qkv[2] = 0.0
    qkv[3, hq:, 5] = np.inf
    qkv[5, hq:, 6] = -np.inf
    qkv[6, hq:, 7] = np.nan
    state = fp8_state(rng, nb, hkv, bs, d)
    cs = pa.rope_table(maxp, rot).numpy()
    q, k, v = dev(qkv, dtype).split([hq, hkv, hkv], 1)
    kc, ks, vc, vs = f8(state[0]), dev(state[1]), f8(state[2]), dev(state[3])
    pa.device_status(clear=True)
    left_out = slots.copy()
    if rope:
        q_out = torch.full((T, hq, d), 7.0, dtype=TORCH_DT[dtype], device="cuda")
        pa.rope_write_kv_fp8(q, k, v, kc, vc, ks, vs, dev(slots), dev(pos), dev(cs), interleaved=il, q_out=q_out)
        assert pa.device_status() == pa.DEV_ERR_SLOT | pa.DEV_ERR_POSITION
        p = np.clip(pos, 0, maxp - 1)
        want = round_to(R.rotate(qkv[:, :hq], cs, p, il), dtype)
        want[7], want[11] = 7.0, 0.0
        assert np.array_equal(q_out.float().cpu().numpy(), want)
        kt = R.rotate(qkv[:, hq:hq + hkv], cs, p, il)
        left_out[[7, 11]] = -1
    else:
        pa.write_kv_fp8(k, v, kc, vc, ks, vs, dev(slots))
        assert pa.device_status() == pa.DEV_ERR_SLOT
        kt = qkv[:, hq:hq + hkv]
    kb, kss, vb, vss = (x.copy() for x in state)
    R.append_rows(kt, kb, kss, left_out)
    R.append_rows(qkv[:, hq + hkv:], vb, vss, left_out)
    check_fp8(kc, ks, vc, vs, (kb, kss, vb, vss))


@pytest.mark.parametrize("bs,d", [(16, 64), (32, 128)])
def test_append_fp8_many_tokens_per_warp(bs, d):
    """A long chunked prefill: warps own block_size tokens, runs start anywhere and cross the warps' stretches."""
    require_gpu()
    rng = np.random.default_rng(bs)
    hkv, T = 32, 0
    lens = [1, 5, 333, 700, 17, bs, 2 * bs, 129]
    nb = sum(-(-(n + bs) // bs) for n in lens) + 4
    slots, _ = token_mix(rng, nb, bs, 0, [(int(rng.integers(0, bs)), n) for n in lens])
    T = len(slots)
    assert T * 2 * hkv > 148 * 64 * 4  # the launch that gives a warp block_size tokens
    kv = rows(rng, "bf16", T, 2 * hkv, d)
    state = fp8_state(rng, nb, hkv, bs, d)
    kc, ks, vc, vs = f8(state[0]), dev(state[1]), f8(state[2]), dev(state[3])
    k, v = dev(kv, "bf16").split([hkv, hkv], 1)
    pa.write_kv_fp8(k, v, kc, vc, ks, vs, dev(slots))
    kb, kss, vb, vss = (x.copy() for x in state)
    R.append_rows(kv[:, :hkv], kb, kss, slots)
    R.append_rows(kv[:, hkv:], vb, vss, slots)
    check_fp8(kc, ks, vc, vs, (kb, kss, vb, vss))
    assert pa.device_status() == 0


def test_append_fp8_run_stretched_by_skipped_tokens():
    """Skipped tokens inside, before and behind a block's tokens, in numbers that pass a warp's windows."""
    require_gpu()
    rng = np.random.default_rng(21)
    hkv, d, bs, nb = 2, 128, 16, 8
    for gaps in ([0, 3, 40, 0, 70], [33, 0, 1, 31, 5]):
        slots = []
        for i, gap in enumerate(gaps):
            slots += [-1] * gap + [2 * bs + 3 + 2 * i, 2 * bs + 4 + 2 * i]
        slots += [-1] * 9 + [5 * bs] + [-1] * 50 + [5 * bs + 1, 0]
        slots = np.array(slots, np.int64)
        kv = rows(rng, "fp16", len(slots), 2 * hkv, d, gain=3.0)
        state = fp8_state(rng, nb, hkv, bs, d)
        kc, ks, vc, vs = f8(state[0]), dev(state[1]), f8(state[2]), dev(state[3])
        k, v = dev(kv, "fp16").split([hkv, hkv], 1)
        pa.write_kv_fp8(k, v, kc, vc, ks, vs, dev(slots))
        kb, kss, vb, vss = (x.copy() for x in state)
        R.append_rows(kv[:, :hkv], kb, kss, slots)
        R.append_rows(kv[:, hkv:], vb, vss, slots)
        check_fp8(kc, ks, vc, vs, (kb, kss, vb, vss))
    assert pa.device_status() == 0


def test_append_fp8_token_by_token_grows_scales_and_foreign_scales_stand():
    """One call per token, magnitudes rising and falling; blocks that start with a scale of the caller's own (not a
    power of two, zero) keep it while it holds the rows."""
    require_gpu()
    rng = np.random.default_rng(9)
    nb, hkv, bs, d = 6, 3, 16, 64
    state = fp8_state(rng, nb, hkv, bs, d)
    state[1][0], state[3][0] = 0.3, 0.013
    state[1][1], state[3][1] = 0.0, 0.0
    kc, ks, vc, vs = f8(state[0]), dev(state[1]), f8(state[2]), dev(state[3])
    kb, kss, vb, vss = (x.copy() for x in state)
    for step in range(40):
        slots = np.array([b * bs + (step + 1 + 3 * b) % bs for b in range(4)], np.int64)
        kv = rows(rng, "bf16", 4, 2 * hkv, d, gain=2.0 ** rng.integers(-9, 6))
        k, v = dev(kv, "bf16").split([hkv, hkv], 1)
        pa.write_kv_fp8(k, v, kc, vc, ks, vs, dev(slots))
        R.append_rows(kv[:, :hkv], kb, kss, slots)
        R.append_rows(kv[:, hkv:], vb, vss, slots)
        check_fp8(kc, ks, vc, vs, (kb, kss, vb, vss))
    assert pa.device_status() == 0


def test_append_fp8_captured_and_replayed():
    require_gpu()
    rng = np.random.default_rng(11)
    hq, hkv, d, bs, nb, T = 8, 2, 128, 16, 16, 6
    cs = pa.rope_table(128, d, device="cuda")
    kc, vc = (torch.zeros((nb, hkv, bs, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, hkv), device="cuda") for _ in range(2))
    qkv = torch.zeros((T, hq + 2 * hkv, d), dtype=torch.float16, device="cuda")
    slots, pos = (torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2))
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    q_out = torch.zeros((T, hq, d), dtype=torch.float16, device="cuda")
    slots.fill_(-1)
    call = lambda: pa.rope_write_kv_fp8(q, k, v, kc, vc, ks, vs, slots, pos, cs, q_out=q_out)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    kb, vb = (np.zeros((nb, hkv, bs, d), np.uint8) for _ in range(2))
    kss, vss = (np.zeros((nb, hkv), np.float32) for _ in range(2))
    table = cs.cpu().numpy()
    for step in range(20):
        x = rows(rng, "fp16", T, hq + 2 * hkv, d, gain=1 + step)
        s = np.array([2 * t * bs + step % bs for t in range(T)], np.int64)
        s[T - 1] = -1
        p = np.full(T, step, np.int64)
        p[T - 1] = -1
        qkv.copy_(dev(x, "fp16")), slots.copy_(dev(s)), pos.copy_(dev(p))
        graph.replay()
        R.append_rows(R.rotate(x[:, hq:hq + hkv], table, np.maximum(p, 0), False), kb, kss, s)
        R.append_rows(x[:, hq + hkv:], vb, vss, s)
        check_fp8(kc, ks, vc, vs, (kb, kss, vb, vss))
    assert pa.device_status() == 0


def test_refusals():
    require_gpu()
    T, hq, hkv, d, bs, nb = 3, 4, 2, 128, 16, 4
    q, k, v = (torch.zeros((T, h, d), dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv))
    kc, vc = (torch.zeros((nb, hkv, bs, d), dtype=torch.float16, device="cuda") for _ in range(2))
    k8, v8 = (torch.zeros((nb, hkv, bs, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((nb, hkv), device="cuda") for _ in range(2))
    slots, pos = (torch.arange(T, device="cuda") for _ in range(2))
    cs = pa.rope_table(8, d, device="cuda")
    E = pa.PagedAttentionError
    n0 = pa.launch_count()
    bad = [
        lambda: pa.rope_write_kv(q, k, v, k8, v8, slots, pos, cs),             # 8-bit caches, 16-bit call
        lambda: pa.rope_write_kv(q.bfloat16(), k, v, kc, vc, slots, pos, cs),  # another type
        lambda: pa.rope_write_kv(q, k, v, kc, vc, slots, pos.int(), cs),
        lambda: pa.rope_write_kv(q, k, v, kc, vc, slots, pos[:2], cs),
        lambda: pa.rope_write_kv(q, k, v, kc, vc, slots, pos, cs.double()),
        lambda: pa.rope_write_kv(q, k, v, kc, vc, slots, pos, pa.rope_table(8, 24, device="cuda")),
        lambda: pa.rope_write_kv(q, k, v, kc, vc, slots, pos, pa.rope_table(8, 256, device="cuda")),
        lambda: pa.rope_write_kv(q, k, v, kc, vc, slots, pos, cs.cpu()),
        lambda: pa.rope_write_kv(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, kc, vc, slots, pos, cs),
        lambda: pa.rope_write_kv(None, k, v, kc, vc, slots, pos, cs, q_out=q),
        lambda: pa.write_kv_fp8(k, v, kc, vc, ks, vs, slots),
        lambda: pa.write_kv_fp8(k, v, k8, v8, ks.half(), vs, slots),
        lambda: pa.write_kv_fp8(k, v, k8, v8, ks, vs[:2], slots),
        lambda: pa.write_kv_fp8(k.float(), v.float(), k8, v8, ks, vs, slots),
        lambda: pa.write_kv_fp8(k[:2], v, k8, v8, ks, vs, slots),
        lambda: pa.rope_write_kv_fp8(q, k, v, k8, v8, ks, vs.cpu(), slots, pos, cs),
    ]
    for call in bad:
        with pytest.raises(E):
            call()
    assert pa.launch_count() == n0 and pa.device_status() == 0
