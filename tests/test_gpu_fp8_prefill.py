"""Causal prefill over 8-bit caches against the 64-bit reference on the very bytes and scales the kernel reads."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref as R
import paged_kv_cache_457_b200 as pa
from fp8_cases import HALF_STEP, Batch, tolerance
from gpu_util import require_gpu
from test_gpu_fp8_decode import dev, on_gpu, queries

pytestmark = pytest.mark.gpu


def starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def check(got, q, b, new, dtype, scale, kv_half_step=0.0):
    k, v = b.values()
    n = int(sum(new))
    out, mean_abs, dots = R.attention(q.double().numpy()[:n], k, v, b.tables, b.ctx, scale, new=new, bounds=True)
    vs = float(np.nanmax(b.pools[3], initial=0.0))
    keys = np.repeat(b.ctx, new)
    # weights are rounded to the storage type; the running maximum lags the true one by at most 2^8, so the largest
    # weight is at least 1 and fp16's subnormal weights are off by 2^-25 of it (bf16 has none)
    tol = tolerance(out, mean_abs, dots, keys, b.d, dtype, 448.0 * vs, HALF_STEP[dtype],
                    2.0 ** -25 if dtype == "fp16" else 0.0, kv_half_step)
    got = got[:n].double().cpu().numpy()
    assert np.all(np.isfinite(got))
    err = np.abs(got - out)
    worst = float((err / tol).max(initial=0.0))
    assert worst <= 1.0, f"{err.max():.3e} off, {worst:.2f} of the bound"


def run(b, q, new, scale, most=None, **kw):
    kc, vc, ks, vs = on_gpu(b)
    return pa.prefill_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(starts(new)), dev(b.ctx), scale,
                          max(new) if most is None else most, **kw)


CASES = [
    [(70, 70), (200, 33), (9, 9), (1, 1)],
    [(128, 128), (129, 129), (256, 256), (257, 257), (300, 44)],
    [(640, 1), (513, 2), (17, 16), (16, 16), (31, 15), (0, 0), (5, 0)],
    [(700, 300), (0, 0), (520, 520)],
    [(1030, 17), (33, 33), (400, 5)],
]
HEADS = [(4, 2, 64, 16), (8, 8, 128, 16), (8, 1, 128, 32), (6, 2, 64, 32), (3, 3, 128, 16)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", HEADS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_reference(dtype, hq, hkv, d, bs, case):
    require_gpu()
    rng = np.random.default_rng(case * 11 + d + bs)
    ctx, new = [c for c, _ in CASES[case]], [n for _, n in CASES[case]]
    b = Batch(rng, ctx, hkv, d, bs)
    q = queries(rng, dtype, sum(new), hq, d)
    out = run(b, q, new, d ** -0.5)
    check(out, q, b, new, dtype, d ** -0.5)
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("new", [1, 2, 5, 16, 17, 24, 25, 40])
def test_few_tokens_behind_long_contexts(dtype, new):
    require_gpu()
    rng = np.random.default_rng(new)
    counts = [new, max(1, new - 1), new, 1, 0, new]
    ctx = [900, 64, new, 333, 50, 2100]
    b = Batch(rng, ctx, 2, 128, 16)
    q = queries(rng, dtype, sum(counts), 8, 128)
    out = run(b, q, counts, 0.0884)
    check(out, q, b, counts, dtype, float(np.float32(0.0884)))
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(7, 1, 128, 16), (3, 3, 64, 32), (16, 1, 64, 16), (5, 5, 128, 32), (11, 1, 128, 16),
                                         (12, 2, 64, 16), (32, 4, 128, 16)])
@pytest.mark.parametrize("ctx0", [0, 90, 1500])
def test_few_tokens_of_every_grouping(dtype, hq, hkv, d, bs, ctx0):
    """Row groups of one to eight tokens; tables wide enough for the split kernel, and narrow ones for the other."""
    require_gpu()
    rng = np.random.default_rng(hq + ctx0)
    new = [9, 1, 0, 4, 7, 2]
    b = Batch(rng, [n + ctx0 + i * 17 if n else 40 for i, n in enumerate(new)], hkv, d, bs, width=500 if ctx0 else None)
    q = queries(rng, dtype, sum(new), hq, d)
    out = run(b, q, new, d ** -0.5)
    check(out, q, b, new, dtype, d ** -0.5)
    assert pa.device_status() == 0


@pytest.mark.parametrize("new", [[6, 3], [150, 40]])
def test_nan_stays_its_own(new):
    """A query row of NaN, and a sequence whose values are NaN: the other rows are as before."""
    require_gpu()
    rng = np.random.default_rng(38)
    b = Batch(rng, [n + 50 for n in new], 2, 64, 16)
    q = queries(rng, "bf16", sum(new), 4, 64)
    good = run(b, q, new, 0.125)
    q2 = q.clone()
    q2[1, 2] = float("nan")
    out = run(b, q2, new, 0.125)
    same = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    same[1, 2] = False
    assert torch.equal(out[same], good[same]) and torch.isnan(out[1, 2]).all()
    b.pools[2][b.tables[1, 0]] = 0x7F
    out = run(b, q, new, 0.125)
    assert torch.equal(out[:new[0]], good[:new[0]]) and torch.isnan(out[new[0]:]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("new", [[6, 3], [150, 40]])
def test_scales_that_are_no_powers_of_two(dtype, new):
    require_gpu()
    rng = np.random.default_rng(31)
    b = Batch(rng, [400, 77], 2, 64, 16, spread=4.0, foreign=True)
    q = queries(rng, dtype, sum(new), 4, 64, gain=0.5)
    check(run(b, q, new, 0.125), q, b, new, dtype, 0.125, kv_half_step=HALF_STEP[dtype])


@pytest.mark.parametrize("new", [[3, 4], [100, 50]])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_any_finite_scale(scale, new):
    require_gpu()
    rng = np.random.default_rng(32)
    b = Batch(rng, [200, 77], 2, 64, 16)
    q = queries(rng, "bf16", sum(new), 4, 64)
    check(run(b, q, new, scale), q, b, new, "bf16", float(np.float32(scale)))


@pytest.mark.parametrize("new", [[7, 0, 4], [300, 0, 130]])
def test_strided_rows_and_rows_behind_the_last_sequence(new):
    require_gpu()
    rng = np.random.default_rng(33)
    hq, hkv, d = 4, 2, 128
    ctx = [n + 60 for n in new]
    b = Batch(rng, ctx, hkv, d, 16, width=40)
    N = sum(new) + 9  # rows behind the last sequence
    rows = queries(rng, "bf16", N, hq + 2, d)
    out = torch.full((N, hq + 1, d), 5.0, dtype=torch.bfloat16, device="cuda")
    kc, vc, ks, vs = on_gpu(b)
    got = pa.prefill_fp8(rows.cuda()[:, 1:hq + 1], kc, vc, ks, vs, dev(b.tables), dev(starts(new)), dev(b.ctx), 0.09,
                         max(new) + 3, out=out[:, :hq])
    check(got, rows[:, 1:hq + 1], b, new, "bf16", float(np.float32(0.09)))
    assert torch.all(out[sum(new):] == 5.0) and torch.all(out[:, hq] == 5.0)
    assert pa.device_status() == 0


@pytest.mark.parametrize("new", [[5, 8, 6, 3], [60, 270, 130, 40]])
def test_device_side_errors(new):
    require_gpu()
    rng = np.random.default_rng(34)
    hq, hkv, d, bs = 4, 2, 128, 16
    ctx = [n + 90 for n in new]
    b = Batch(rng, ctx, hkv, d, bs)
    q = queries(rng, "fp16", sum(new), hq, d).cuda()
    kc, vc, ks, vs = on_gpu(b)
    st = dev(starts(new))
    at = starts(new)

    def call(tables=b.tables, c=b.ctx, s=st, most=max(new)):
        out = torch.full((sum(new), hq, d), 7.0, dtype=torch.float16, device="cuda")
        pa.prefill_fp8(q, kc, vc, ks, vs, dev(tables), s, dev(c), 0.09, most, out=out)
        return out

    good = call()
    assert pa.device_status() == 0
    others = [i for i in range(sum(new)) if not at[1] <= i < at[2]]
    for bad_id in (-1, kc.shape[0]):
        for col in (0, (ctx[1] - 1) // bs):
            t = b.tables.copy()
            t[1, col] = bad_id
            out = call(tables=t)
            assert pa.device_status() == pa.DEV_ERR_BLOCK_ID
            assert torch.equal(out[others], good[others])
            last = out[at[2] - 1]  # the last token needs every block
            assert torch.all(last == 0)
            if col == 0:
                assert torch.all(out[at[1]:at[2]] == 0)
    c = b.ctx.copy()
    c[1] = new[1] - 1  # fewer tokens than it brings
    out = call(c=c)
    assert pa.device_status() == pa.DEV_ERR_CONTEXT
    assert torch.all(out[at[1]:at[2]] == 0) and torch.equal(out[others], good[others])
    c[1] = b.tables.shape[1] * bs + 1
    out = call(c=c)
    assert pa.device_status() == pa.DEV_ERR_CONTEXT and torch.all(out[at[1]:at[2]] == 0)
    s = at.copy()
    s[4] = sum(new) + 1  # the last sequence leaves the rows
    out = call(s=dev(s))
    assert pa.device_status() == pa.DEV_ERR_CONTEXT
    assert torch.all(out[at[3]:] == 7.0) and torch.equal(out[:at[3]], good[:at[3]])


def test_max_query_len_too_small_is_flagged():
    require_gpu()
    rng = np.random.default_rng(35)
    for new, most, written in (([300, 4], 256, 256), ([9, 2], 4, None)):
        b = Batch(rng, [n + 20 for n in new], 2, 64, 16)
        q = queries(rng, "fp16", sum(new), 4, 64)
        out = run(b, q, new, 0.125, most=most)
        assert pa.device_status() & pa.DEV_ERR_CONTEXT_HINT or written is None
        k, v = b.values()
        ref = R.attention(q.double().numpy(), k, v, b.tables, b.ctx, 0.125, new=new)
        rows = list(range(min(new[0], written or most))) + list(range(new[0], sum(new)))
        assert np.abs(out.double().cpu().numpy()[rows] - ref[rows]).max() < 1e-2


@pytest.mark.parametrize("new", [[5, 2], [200, 90]])
def test_graphs_beside_each_other(new):
    require_gpu()
    rng = np.random.default_rng(36)
    b = Batch(rng, [n + 700 for n in new], 4, 128, 16)
    kc, vc, ks, vs = on_gpu(b)
    t, c, s = dev(b.tables), dev(b.ctx), dev(starts(new))
    qs = [queries(rng, "bf16", sum(new), 16, 128).cuda() for _ in range(3)]
    call = lambda q: pa.prefill_fp8(q, kc, vc, ks, vs, t, s, c, 0.09, max(new))  # noqa: E731
    want = [call(q) for q in qs]
    graphs, outs = [], []
    for q in qs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(q))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager = call(qs[2])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[2])
    assert pa.device_status() == 0


def test_refusals_and_empty_calls():
    require_gpu()
    rng = np.random.default_rng(37)
    b = Batch(rng, [20, 30], 2, 64, 16)
    q = queries(rng, "fp16", 12, 4, 64).cuda()
    kc, vc, ks, vs = on_gpu(b)
    t, c, s = dev(b.tables), dev(b.ctx), dev(starts([5, 7]))
    n0 = pa.launch_count()
    bad = [
        lambda: pa.prefill_fp8(q.float(), kc, vc, ks, vs, t, s, c, 0.1, 7),
        lambda: pa.prefill_fp8(q, kc.half(), vc.half(), ks, vs, t, s, c, 0.1, 7),
        lambda: pa.prefill_fp8(q, kc, vc, ks[:1], vs, t, s, c, 0.1, 7),
        lambda: pa.prefill_fp8(q, kc, vc, ks, vs, t, s[:2], c, 0.1, 7),
        lambda: pa.prefill_fp8(q, kc, vc, ks, vs, t, s.long(), c, 0.1, 7),
        lambda: pa.prefill_fp8(q[:, :3], kc, vc, ks, vs, t, s, c, 0.1, 7),
        lambda: pa.prefill_fp8(q, kc, vc, ks, vs, t, s, c, float("nan"), 7),
        lambda: pa.prefill_fp8(q, kc, vc, ks, vs, t, s, c, 0.1, -1),
        lambda: pa.prefill_fp8(q, kc, vc, ks, vs, t, s, c, 0.1, 7, out=q[:, :2]),
    ]
    for call in bad:
        with pytest.raises(pa.PagedAttentionError):
            call()
    assert pa.prefill_fp8(q[:0], kc, vc, ks, vs, t, s, c, 0.1, 7).shape == (0, 4, 64)
    out = torch.full_like(q, 3.0)
    pa.prefill_fp8(q, kc, vc, ks, vs, t, s, c, 0.1, 0, out=out)
    assert torch.all(out == 3.0)
    assert pa.launch_count() == n0 and pa.device_status() == 0
