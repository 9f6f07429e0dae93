"""Decode attention over 8-bit caches against the 64-bit reference on the very bytes and scales the kernel reads."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref as R
import paged_kv_cache_457_b200 as pa
from fp8_cases import Batch, tolerance
from gpu_util import TORCH_DT, require_gpu

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def on_gpu(b):
    kb, ks, vb, vs = b.pools
    return dev(kb).view(torch.float8_e4m3fn), dev(vb).view(torch.float8_e4m3fn), dev(ks), dev(vs)


def queries(rng, dtype, *shape, gain=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * gain).astype(np.float32)).to(TORCH_DT[dtype])


def check(got, q, b, dtype, scale):
    k, v = b.values()
    out, mean_abs, dots = R.attention(q.double().numpy(), k, v, b.tables, b.ctx, scale, bounds=True)
    vs = float(np.nanmax(b.pools[3], initial=0.0))
    tol = tolerance(out, mean_abs, dots, b.ctx, b.d, dtype, 448.0 * vs)
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    err = np.abs(got - out)
    worst = float((err / tol).max(initial=0.0))
    assert worst <= 1.0, f"{err.max():.3e} off, {worst:.2f} of the bound"
    assert np.all(got[b.ctx == 0] == 0)


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 47, 64, 65, 200, 513, 0, 1000]
SHAPES = [(8, 8, 64, 16), (32, 8, 128, 16), (12, 4, 128, 32), (16, 1, 128, 16), (7, 1, 64, 32), (5, 5, 64, 16), (16, 8, 128, 32),
          (11, 1, 128, 16)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
@pytest.mark.parametrize("part", [0, 16, 128])
def test_small_shapes(dtype, hq, hkv, d, bs, part):
    require_gpu()
    rng = np.random.default_rng(hq * 7 + d + bs)
    b = Batch(rng, LENS, hkv, d, bs)
    q = queries(rng, dtype, len(LENS), hq, d)
    kc, vc, ks, vs = on_gpu(b)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), d ** -0.5, max_context_len=1000,
                        partition_tokens=part)
    check(out, q, b, dtype, d ** -0.5)
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("spread,foreign", [(2.0 ** 6, False), (2.0 ** 12, True), (1.0, True)])
def test_scales_far_apart_and_no_powers_of_two(dtype, spread, foreign):
    require_gpu()
    rng = np.random.default_rng(17)
    b = Batch(rng, [700, 33, 5, 256], 2, 128, 16, spread=spread, foreign=foreign)
    if dtype == "fp16":  # outputs have to fit the type
        b.pools[3] = b.pools[3] * np.float32(2.0 ** -3)
    q = queries(rng, dtype, 4, 8, 128, gain=1.0 / spread)
    kc, vc, ks, vs = on_gpu(b)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.1, max_context_len=700)
    check(out, q, b, dtype, 0.1)
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_zero_blocks_and_zero_scales(dtype):
    require_gpu()
    rng = np.random.default_rng(18)
    b = Batch(rng, [40, 16, 100], 2, 64, 16)
    kb, ks_, vb, vs_ = b.pools
    t = b.tables
    vb[t[0, 0]], vs_[t[0, 0]] = 0, 0.0
    kb[t[0, 1]], ks_[t[0, 1]] = 0, 0.0
    vb[t[1, 0]], vs_[t[1, 0]] = 0, 2.0 ** -64  # a sequence whose values are all zero
    q = queries(rng, dtype, 3, 4, 64)
    kc, vc, ks, vs = on_gpu(b)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.125, max_context_len=100)
    check(out, q, b, dtype, 0.125)
    assert torch.all(out[1] == 0)


@pytest.mark.parametrize("gain", [1e-30, 1e-6, 30.0, 1e4])
def test_query_magnitudes(gain):
    """bf16 rows far from fp16's range: scaled by a power of two on the way, without loss."""
    require_gpu()
    rng = np.random.default_rng(19)
    b = Batch(rng, [300, 77], 2, 128, 16)
    q = queries(rng, "bf16", 2, 8, 128, gain=gain)
    q[0, 1] = 0
    kc, vc, ks, vs = on_gpu(b)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.0883, max_context_len=300)
    check(out, q, b, "bf16", float(np.float32(0.0883)))


@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_any_finite_scale_and_a_nan_row(scale, part):
    require_gpu()
    rng = np.random.default_rng(26)
    b = Batch(rng, [200, 77, 31], 2, 64, 16)
    q = queries(rng, "bf16", 3, 4, 64)
    kc, vc, ks, vs = on_gpu(b)
    call = lambda x: pa.decode_fp8(x.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), scale, 200, partition_tokens=part)  # noqa: E731
    good = call(q)
    check(good, q, b, "bf16", float(np.float32(scale)))
    q[1, 2] = float("nan")
    out = call(q)
    same = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    same[1, 2] = False
    assert torch.equal(out[same], good[same]) and torch.isnan(out[1, 2]).all()


def test_tables_cut_from_wider_ones():
    require_gpu()
    rng = np.random.default_rng(27)
    b = Batch(rng, [100, 0, 64], 2, 64, 16, width=13)
    q = queries(rng, "fp16", 3, 4, 64)
    kc, vc, ks, vs = on_gpu(b)
    t = dev(b.tables)
    want = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, t, dev(b.ctx), 0.125, 100)
    assert torch.equal(pa.decode_fp8(q.cuda(), kc, vc, ks, vs, t[:, :7], dev(b.ctx), 0.125, 100), want)
    one = pa.decode_fp8(q.cuda()[:1], kc, vc, ks, vs, t[:1, :7], dev(b.ctx[:1]), 0.125, 100)
    assert torch.equal(one, want[:1])
    check(want, q, b, "fp16", 0.125)


def test_sharp_weights_and_a_rising_maximum():
    """Keys that raise the maximum again and again, and one token that takes all the weight."""
    require_gpu()
    rng = np.random.default_rng(20)
    hkv, d, bs, L = 1, 64, 16, 640
    b = Batch(rng, [L], hkv, d, bs)
    x = rng.standard_normal((b.pools[0].shape[0], hkv, bs, d)).astype(np.float32) * 0.1
    for i in range(L // bs):
        x[b.tables[0, i], 0, :, 0] = i * 4.0
    b.pools[0], b.pools[1] = R.quantise_pool(x)
    q = torch.zeros((1, 4, d), dtype=torch.float16)
    q[0, :, 0] = torch.tensor([1.0, -1.0, 8.0, -8.0])
    kc, vc, ks, vs = on_gpu(b)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.5, max_context_len=L)
    check(out, q, b, "fp16", 0.5)


def test_long_context_many_pieces():
    require_gpu()
    rng = np.random.default_rng(21)
    b = Batch(rng, [9001, 3, 4097], 2, 128, 32)
    q = queries(rng, "bf16", 3, 8, 128)
    kc, vc, ks, vs = on_gpu(b)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.0884, max_context_len=9001)
    check(out, q, b, "bf16", float(np.float32(0.0884)))
    again = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.0884)  # the bound read back
    assert torch.equal(out, again)


def test_many_sequences_strided_rows_and_wide_tables():
    require_gpu()
    rng = np.random.default_rng(22)
    S, hq, hkv, d, bs = 3006, 4, 2, 64, 16
    b = Batch(rng, rng.integers(0, 40, S), hkv, d, bs, width=9)
    rows = queries(rng, "fp16", S, hq + 3, d)
    q = rows.cuda()[:, :hq]
    out = torch.full((S, hq + 1, d), 5.0, dtype=torch.float16, device="cuda")
    kc, vc, ks, vs = on_gpu(b)
    pa.decode_fp8(q, kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.125, max_context_len=39, out=out[:, :hq])
    check(out[:, :hq], rows[:, :hq], b, "fp16", 0.125)
    assert torch.all(out[:, hq] == 5.0)
    assert pa.device_status() == 0


def test_device_side_errors():
    require_gpu()
    rng = np.random.default_rng(23)
    b = Batch(rng, [100, 50, 64, 33], 2, 128, 16)
    q = queries(rng, "fp16", 4, 8, 128)
    kc, vc, ks, vs = on_gpu(b)
    good = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.1, max_context_len=100)
    assert pa.device_status() == 0
    for bad_id in (-1, kc.shape[0]):
        for col in (0, 1, 2):  # first and second half of a tile; the last block of 33 tokens
            t = b.tables.copy()
            t[3, col] = bad_id
            out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(t), dev(b.ctx), 0.1, max_context_len=100)
            assert pa.device_status() == pa.DEV_ERR_BLOCK_ID
            assert torch.all(out[3] == 0) and torch.equal(out[:3], good[:3])
    ctx = b.ctx.copy()
    ctx[1] = b.tables.shape[1] * 16 + 1
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(ctx), 0.1, max_context_len=200)
    assert pa.device_status() == pa.DEV_ERR_CONTEXT and torch.all(out[1] == 0) and torch.equal(out[2:], good[2:])
    ctx[1] = -1
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(ctx), 0.1, max_context_len=100)
    assert pa.device_status() == pa.DEV_ERR_CONTEXT and torch.all(out[1] == 0)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.1, max_context_len=99)
    assert pa.device_status() == pa.DEV_ERR_CONTEXT_HINT and torch.all(out[0] == 0) and torch.equal(out[1:], good[1:])


def test_two_graphs_replayed_on_two_streams_at_once():
    """Each capture holds a workspace of its own: replays beside each other and beside eager calls do not disturb."""
    require_gpu()
    rng = np.random.default_rng(24)
    b = Batch(rng, [3000, 1500, 10, 700], 4, 128, 16)
    kc, vc, ks, vs = on_gpu(b)
    tables, ctx = dev(b.tables), dev(b.ctx)
    qs = [queries(rng, "bf16", 4, 16, 128).cuda() for _ in range(3)]
    want = [pa.decode_fp8(q, kc, vc, ks, vs, tables, ctx, 0.09, max_context_len=3000) for q in qs]
    graphs, outs = [], []
    for q in qs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pa.decode_fp8(q, kc, vc, ks, vs, tables, ctx, 0.09, max_context_len=3000))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = pa.decode_fp8(qs[2], kc, vc, ks, vs, tables, ctx, 0.09, max_context_len=3000)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[2])
    assert pa.device_status() == 0


def test_refusals_and_empty_batch():
    require_gpu()
    rng = np.random.default_rng(25)
    b = Batch(rng, [20, 30], 2, 64, 16)
    q = queries(rng, "fp16", 2, 4, 64).cuda()
    kc, vc, ks, vs = on_gpu(b)
    t, c = dev(b.tables), dev(b.ctx)
    E = pa.PagedAttentionError
    n0 = pa.launch_count()
    bad = [
        lambda: pa.decode_fp8(q.float(), kc, vc, ks, vs, t, c, 0.1, 30),
        lambda: pa.decode_fp8(q, kc.half(), vc.half(), ks, vs, t, c, 0.1, 30),
        lambda: pa.decode_fp8(q, kc, vc, ks.double(), vs, t, c, 0.1, 30),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs.t().contiguous(), t, c, 0.1, 30),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs, t.long(), c, 0.1, 30),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs, t, c.cpu(), 0.1, 30),
        lambda: pa.decode_fp8(q[:, :3], kc, vc, ks, vs, t, c, 0.1, 30),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs, t, c, float("inf"), 30),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs, t, c, 0.1, 30, partition_tokens=8),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs, t, c, 0.1, -1),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs, t, c, 0.1, 30, out=q[:, :2]),
        lambda: pa.decode_fp8(q, kc, vc, ks, vs, t, c, 0.1, 30, partition_tokens=32,
                              workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(E):
            call()
    assert pa.decode_fp8(q[:0], kc, vc, ks, vs, t[:0], c[:0], 0.1).shape == (0, 4, 64)
    assert pa.launch_count() == n0 and pa.device_status() == 0
