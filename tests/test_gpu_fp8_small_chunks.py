"""The smallest cuts of the 8-bit split decode, with many more chunks than warps: every warp takes chunk after chunk."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_cache_457_b200 as pa
from fp8_cases import Batch
from gpu_util import require_gpu
from test_gpu_fp8_decode import check, dev, on_gpu, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("part", [16, 32, 48, 64, 80])
@pytest.mark.parametrize("dtype,hq,hkv,d,bs,seqs,longest", [("fp16", 26, 2, 64, 16, 30, 500), ("bf16", 32, 32, 64, 32, 138, 10),
                                                            ("fp16", 5, 5, 128, 32, 20, 3000)])
def test_many_small_chunks(part, dtype, hq, hkv, d, bs, seqs, longest):
    require_gpu()
    rng = np.random.default_rng(seqs)
    ctx = rng.integers(0, longest + 1, seqs)
    b = Batch(rng, ctx, hkv, d, bs)
    q = queries(rng, dtype, seqs, hq, d)
    kc, vc, ks, vs = on_gpu(b)
    call = lambda: pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), d ** -0.5,  # noqa: E731
                                 max_context_len=longest, partition_tokens=part)
    out = call()
    assert pa.device_status() == 0
    check(out, q, b, dtype, d ** -0.5)
    for _ in range(5):
        assert torch.equal(call(), out)
