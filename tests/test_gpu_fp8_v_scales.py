"""V scales at the ends of what the header allows, on every kernel that reads them: per-unit and split decode, the same
for prefill calls of few tokens, and the 128-row tiles.

Powers of two move through the arithmetic exactly, so caches whose V scales are 2^-70 (bf16 holds such outputs as normal
numbers) are checked in units of 2^-70, against the bounds that hold for ordinary scales."""
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

PATHS = ["unit", "split", "few unit", "few split", "tiles"]
CTX = [333, 47, 160]


def batch(rng, path):
    return Batch(rng, CTX, 2, 64, 16, width=1000 if path == "few split" else None)


def attend(path, b, q, new):
    kc, vc, ks, vs = on_gpu(b)
    if path in ("unit", "split"):
        out = pa.decode_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(b.ctx), 0.125, max(CTX),
                            partition_tokens=64 if path == "split" else 0)
    else:
        out = pa.prefill_fp8(q.cuda(), kc, vc, ks, vs, dev(b.tables), dev(starts(new)), dev(b.ctx), 0.125, max(new))
    assert pa.device_status() == 0
    return out


def tokens(path):
    return {"unit": [1, 1, 1], "split": [1, 1, 1], "tiles": [30, 26, 40]}.get(path, [5, 9, 1])


def check(path, out, q, b, new):
    if path in ("unit", "split"):
        check_decode(out, q, b, "bf16", 0.125)
    else:
        check_prefill(out, q, b, new, "bf16", 0.125)


@pytest.mark.parametrize("path", PATHS)
def test_small_scales(path):
    require_gpu()
    rng = np.random.default_rng(61)
    new = tokens(path)
    b, q = batch(rng, path), queries(rng, "bf16", sum(tokens(path)), 8, 64)
    b.pools[3] = b.pools[3] * np.float32(2.0 ** -70)
    out = attend(path, b, q, new).float() * 2.0 ** 70
    b.pools[3] = b.pools[3] * np.float32(2.0 ** 70)
    check(path, out, q, b, new)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("unit", [0, -70, 40])
def test_blocks_of_scale_zero_whatever_their_bytes(path, unit):
    """Every third block has scale 0 over random bytes: its tokens take weight and give nothing.  One sequence has no
    other blocks: its rows are zeros."""
    require_gpu()
    rng = np.random.default_rng(62)
    new = tokens(path)
    b, q = batch(rng, path), queries(rng, "bf16", sum(tokens(path)), 8, 64)
    for s, n in enumerate(b.ctx):
        ids = b.tables[s, :-(-int(n) // 16)]
        b.pools[3][ids if s == 1 else ids[::3]] = 0.0
    b.pools[3] = b.pools[3] * np.float32(2.0 ** unit)
    out = attend(path, b, q, new).float() * 2.0 ** -unit
    b.pools[3] = b.pools[3] * np.float32(2.0 ** -unit)
    check(path, out, q, b, new)
    assert torch.all(out[new[0]:new[0] + new[1]] == 0)


@pytest.mark.parametrize("path", PATHS)
def test_blocks_of_zeros_beside_very_large_values(path):
    """The appends give a block of zeros the scale 2^-64; its tokens keep their weight beside values of 2^100."""
    require_gpu()
    rng = np.random.default_rng(63)
    new = tokens(path)
    b, q = batch(rng, path), queries(rng, "bf16", sum(tokens(path)), 8, 64)
    b.pools[3] = b.pools[3] * np.float32(2.0 ** 100)
    zeros = np.concatenate([b.tables[s, :-(-int(n) // 16)][1::2] for s, n in enumerate(b.ctx)])
    live = b.pools[2][zeros] != 0x7F
    b.pools[2][zeros] = np.where(live, 0, 0x7F)
    b.pools[3][zeros] = np.float32(2.0 ** -64)
    out = attend(path, b, q, new).float() * 2.0 ** -100
    b.pools[3] = b.pools[3] * np.float32(2.0 ** -100)
    check(path, out, q, b, new)
