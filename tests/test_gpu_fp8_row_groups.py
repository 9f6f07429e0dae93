"""Prefill calls of few tokens per sequence on the split kernel, whose row groups of one sequence share its table row:
contexts short beside the table, so that one warp's stretch of the tile stream holds several groups, and a later group
may need a block that the one before it did not."""
from __future__ import annotations

import numpy as np
import pytest

import paged_kv_cache_457_b200 as pa
from fp8_cases import Batch
from gpu_util import require_gpu
from test_gpu_fp8_decode import queries
from test_gpu_fp8_prefill import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("seqs,longest,new,hq,hkv", [(64, 500, 9, 32, 8), (128, 200, 24, 16, 1)])
def test_groups_of_one_sequence_behind_each_other(dtype, bs, seqs, longest, new, hq, hkv):
    require_gpu()
    rng = np.random.default_rng(seqs + bs)
    d = 128
    ctx = rng.integers(max(20, new), longest + 1, seqs)
    b = Batch(rng, ctx, hkv, d, bs, width=8192 // bs)
    counts = [new] * seqs
    q = queries(rng, dtype, sum(counts), hq, d)
    out = run(b, q, counts, d ** -0.5)
    assert pa.device_status() == 0
    check(out, q, b, counts, dtype, d ** -0.5)
