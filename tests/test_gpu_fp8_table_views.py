"""Block tables that are views ending at the right edge of a wider one, the last row with an odd number of blocks: the
last entry in use is the last of the storage, and nothing behind it may be read (the index-checked build looks)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_cache_457_b200 as pa
from fp8_cases import Batch
from gpu_util import require_gpu
from test_gpu_fp8_decode import check as check_decode
from test_gpu_fp8_decode import dev, on_gpu, queries
from test_gpu_fp8_prefill import check as check_prefill
from test_gpu_fp8_prefill import starts

pytestmark = pytest.mark.gpu


def right_edge(tables, left=6):
    wide = torch.full((tables.shape[0], left + tables.shape[1]), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, left:] = dev(tables)
    view = wide[:, left:]
    end = view.storage_offset() + (view.shape[0] - 1) * view.stride(0) + view.shape[1]
    assert end == wide.numel()  # the view's last entry is the storage's
    return view


@pytest.mark.parametrize("bs,last", [(16, 7 * 16), (16, 6 * 16 + 1), (32, 3 * 32 - 5)])
@pytest.mark.parametrize("part", [0, 32])
def test_decode(bs, last, part):
    require_gpu()
    rng = np.random.default_rng(last)
    ctx = [40, 0, last]
    b = Batch(rng, ctx, 2, 64, bs)
    q = queries(rng, "bf16", 3, 4, 64)
    kc, vc, ks, vs = on_gpu(b)
    view = right_edge(b.tables)
    out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, view, dev(b.ctx), 0.125, max_context_len=max(ctx),
                        partition_tokens=part)
    assert pa.device_status() == 0
    check_decode(out, q, b, "bf16", 0.125)
    assert torch.equal(out, pa.decode_fp8(q.cuda(), kc, vc, ks, vs, view.contiguous(), dev(b.ctx), 0.125,
                                          max_context_len=max(ctx), partition_tokens=part))


@pytest.mark.parametrize("left", [6, 700])  # the stride chooses between the kernels for few tokens
@pytest.mark.parametrize("new", [[9, 0, 5], [100, 3, 40]])
def test_prefill(new, left):
    require_gpu()
    rng = np.random.default_rng(left)
    ctx = [70, 30, 7 * 16] if new[0] == 9 else [105, 30, 7 * 16]
    b = Batch(rng, ctx, 2, 64, 16)  # seven entries a row, all of the last one's in use
    q = queries(rng, "fp16", sum(new), 4, 64)
    kc, vc, ks, vs = on_gpu(b)
    out = pa.prefill_fp8(q.cuda(), kc, vc, ks, vs, right_edge(b.tables, left), dev(starts(new)), dev(b.ctx), 0.125,
                         max(new))
    assert pa.device_status() == 0
    check_prefill(out, q, b, new, "fp16", 0.125)
