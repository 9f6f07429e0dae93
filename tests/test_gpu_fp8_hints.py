"""A max_query_len below a sequence's new tokens sets the hint bit, and only that, on each kernel that prefill_fp8 takes;
rows up to it are as they should be."""
from __future__ import annotations

import numpy as np
import pytest

import fp8_ref as R
import paged_kv_cache_457_b200 as pa
from fp8_cases import HALF_STEP, Batch, tolerance
from gpu_util import require_gpu
from test_gpu_fp8_decode import queries
from test_gpu_fp8_prefill import run, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,most,width", [([9, 2], 4, None), ([9, 2], 4, 600), ([300, 4], 256, None)],
                         ids=["few, per unit", "few, split", "tiles"])
def test_only_the_hint_is_set(new, most, width):
    require_gpu()
    rng = np.random.default_rng(35)
    b = Batch(rng, [n + 20 for n in new], 2, 64, 16, width=width)
    q = queries(rng, "fp16", sum(new), 4, 64)
    out = run(b, q, new, 0.125, most=most)
    assert pa.device_status() == pa.DEV_ERR_CONTEXT_HINT
    k, v = b.values()
    ref, mean_abs, dots = R.attention(q.double().numpy(), k, v, b.tables, b.ctx, 0.125, new=new, bounds=True)
    tol = tolerance(ref, mean_abs, dots, np.repeat(b.ctx, new), b.d, "fp16", 448.0 * float(np.nanmax(b.pools[3])),
                    HALF_STEP["fp16"], 2.0 ** -25)
    at = starts(new)
    rows = [r for s, n in enumerate(new) for r in range(at[s], at[s] + min(n, most))]
    assert np.all(np.abs(out.double().cpu().numpy() - ref)[rows] <= tol[rows])
    run(b, q, new, 0.125, most=max(new))
    assert pa.device_status() == 0
