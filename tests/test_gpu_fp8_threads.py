"""Host threads that call at the same time on one stream, with the workspace that the package keeps for it."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_457_b200 as pa
from fp8_cases import Batch
from gpu_util import require_gpu
from test_gpu_fp8_decode import dev, on_gpu, queries
from test_gpu_fp8_prefill import starts

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream_do_not_mix_their_operations():
    """Prefill (a cleared counter, then the kernel) and split decode (the stream, then the merge), 8-bit and 16-bit."""
    require_gpu()
    rng = np.random.default_rng(51)
    jobs = []
    for ctx, new in (([300, 70, 200], [140, 70, 33]), ([90, 400], [90, 300])):
        b = Batch(rng, ctx, 2, 128, 16)
        args = (queries(rng, "bf16", sum(new), 8, 128).cuda(), *on_gpu(b), dev(b.tables), dev(starts(new)), dev(b.ctx), 0.09)
        jobs.append(lambda a=args, m=max(new): pa.prefill_fp8(*a, m))
    for ctx in ([3000, 10, 500], [40, 2500, 1, 700, 900]):
        b = Batch(rng, ctx, 2, 128, 16)
        q = queries(rng, "bf16", len(ctx), 8, 128).cuda()
        args = (q, *on_gpu(b), dev(b.tables), dev(b.ctx), 0.09)
        jobs.append(lambda a=args, m=max(ctx): pa.decode_fp8(*a, m, partition_tokens=64))
        wide = [torch.randn(b.pools[0].shape, device="cuda").bfloat16() for _ in range(2)]
        args = (q, *wide, dev(b.tables), dev(b.ctx), 0.09)
        jobs.append(lambda a=args, m=max(ctx): pa.decode(*a, m, partition_tokens=64))
    want = [job() for job in jobs]
    again = [job() for job in jobs]
    torch.cuda.synchronize()
    assert pa.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    failed = []

    def work(i):
        for _ in range(60):
            if not torch.equal(jobs[i](), want[i]):
                failed.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, sorted(set(failed))
    assert pa.device_status() == 0
