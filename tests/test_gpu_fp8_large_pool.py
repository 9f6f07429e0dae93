"""Pools whose byte and element offsets pass 32 bits: blocks at the far end are written, read and copied there."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref as R
import paged_kv_cache_457_b200 as pa
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def test_far_blocks_of_a_pool_beyond_4_gib():
    require_gpu()
    hq, hkv, d, bs = 8, 8, 128, 32
    nb = 2 ** 32 // (hkv * bs * d) + 40  # bytes of one 8-bit cache: a little over 4 GiB
    kc, vc = (torch.empty((nb, hkv, bs, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, hkv), device="cuda") for _ in range(2))
    table = pa.rope_table(256, d, device="cuda")
    L = 150
    far = torch.arange(nb - 1, nb - 6, -1, device="cuda")
    near = torch.arange(5, device="cuda")  # where a 32-bit offset would wrap to
    kc.view(torch.uint8)[:40] = 0x11
    vc.view(torch.uint8)[:40] = 0x11
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((L, hq + 2 * hkv, d), generator=g, device="cuda").bfloat16()
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    at = torch.arange(L, device="cuda")
    q = pa.rope_write_kv_fp8(q, k, v, kc, vc, ks, vs, far[at // bs] * bs + at % bs, at, table)
    ctx, tables = torch.tensor([L], dtype=torch.int32, device="cuda"), far.int()[None].contiguous()
    out = pa.prefill_fp8(q, kc, vc, ks, vs, tables, torch.tensor([0, L], dtype=torch.int32, device="cuda"), ctx, 0.09, L)
    last = [pa.decode_fp8(q[-1:], kc, vc, ks, vs, tables, ctx, 0.09, max_context_len=L, partition_tokens=p) for p in (0, 32)]
    pools = [R.values(c.view(torch.uint8)[far].cpu().numpy(), s[far].cpu().numpy()) for c, s in ((kc, ks), (vc, vs))]
    ref = R.attention(q.double().cpu().numpy(), *pools, np.arange(5)[None], [L], float(np.float32(0.09)), new=[L])
    assert np.abs(out.double().cpu().numpy() - ref).max() < 2e-2
    for x in last:
        assert np.abs(x.double().cpu().numpy()[0] - ref[-1]).max() < 2e-2
    pa.copy_blocks_fp8(kc, vc, ks, vs, torch.stack([far, far - 10], 1).contiguous())
    assert torch.equal(kc.view(torch.uint8)[far], kc.view(torch.uint8)[far - 10]) and torch.equal(vs[far], vs[far - 10])
    for c in (kc, vc):
        assert torch.all(c.view(torch.uint8)[near] == 0x11)
    assert pa.device_status() == 0


def test_far_blocks_of_a_16_bit_pool():
    require_gpu()
    hkv, d, bs = 8, 128, 32
    nb = 2 ** 31 // (hkv * bs * d) + 8  # elements pass 2^31
    kc, vc = (torch.empty((nb, hkv, bs, d), dtype=torch.float16, device="cuda") for _ in range(2))
    kc[:8], vc[:8] = 0, 0
    k, v = (torch.randn((3, hkv, d), device="cuda").half() for _ in range(2))
    slots = torch.tensor([nb * bs - 1, (nb - 3) * bs, nb * bs - 40], device="cuda")
    pos = torch.zeros(3, dtype=torch.int64, device="cuda")  # position 0: no turn
    pa.rope_write_kv(None, k, v, kc, vc, slots, pos, pa.rope_table(4, d, device="cuda"))
    assert torch.equal(kc[slots // bs, :, slots % bs], k) and torch.equal(vc[slots // bs, :, slots % bs], v)
    assert torch.all(kc[:8] == 0) and pa.device_status() == 0
