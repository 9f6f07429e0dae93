"""8-bit appends of long inputs: block_size tokens and several heads per warp, the queries in a launch of their own.

Bytes, scales and turned queries are compared for equality, as for short inputs.  The sizes follow the launch rule of
the library: block_size tokens per warp from tokens * pairs > 256 per SM on (pairs: kv heads, for K and for V), and twice
the heads per warp as long as the warps at twice that many heads are at least 32 per SM, up to four."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref as R
import paged_kv_cache_457_b200 as pa
from gpu_util import TORCH_DT, require_gpu
from test_gpu_append import check_fp8, dev, f8, round_to, rows, token_mix

pytestmark = pytest.mark.gpu


def heads_per_warp(T, hkv, bs):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pairs = 2 * hkv
    assert T * pairs > sms * 256
    n = 1
    while n < 4 and -(-T // bs) * (pairs // (2 * n)) >= sms * 32:
        n *= 2
    return n


def prompts(rng, bs, T):
    """About T tokens of prompts and chunks that start anywhere in a block, with gaps of skipped tokens inside blocks."""
    lens = []
    while sum(lens) < T:
        lens.append(int(rng.choice([1, 3, bs - 1, bs, 2 * bs + 5, 200, 701])))
    nb = sum(-(-(n + bs) // bs) for n in lens) + 4
    slots, pos = token_mix(rng, nb, bs, 5, [(int(rng.integers(0, bs)), n) for n in lens])
    out_s, out_p = [], []
    for i, (s, p) in enumerate(zip(slots, pos)):
        if i % 397 == 100:  # a run stretched past its window: skipped tokens between two of a block's
            n = int(rng.choice([1, bs, 40, 75]))
            out_s += [-1] * n
            out_p += list(rng.integers(-1, 50, n))
        out_s.append(s)
        out_p.append(p)
    return nb + 8, np.array(out_s, np.int64), np.array(out_p, np.int64)


def random_state(rng, nb, hkv, bs, d):
    """Bytes of any finite value with power-of-two scales around those of the rows."""
    out = []
    for _ in range(2):
        b = rng.integers(0, 256, (nb, hkv, bs, d), dtype=np.uint8)
        b[(b & 0x7F) == 0x7F] = 0
        out += [b, np.exp2(rng.integers(-10, -4, (nb, hkv))).astype(np.float32)]
    return out


def run(rng, dtype, hq, hkv, d, bs, rot, il, T, want_heads, rope=True, in_place=False, some=False):
    nb, slots, pos = prompts(rng, bs, T)
    T = len(slots)
    assert heads_per_warp(T, hkv, bs) == want_heads
    maxp = int(pos.max()) + 1
    if rope:
        pos[T // 2] = maxp  # out of range: flagged, its K and V skipped, its query zeros
        pos[T // 3] = -1
    slots[T // 4] = nb * bs
    qkv = rows(rng, dtype, T, hq + 2 * hkv, d, gain=2.0)
    qkv[5, hq:, 3] = np.inf
    qkv[9, hq:, 4] = np.nan
    state = random_state(rng, nb, hkv, bs, d)
    kc, ks, vc, vs = f8(state[0]), dev(state[1]), f8(state[2]), dev(state[3])
    q, k, v = dev(qkv, dtype).split([hq, hkv, hkv], 1)
    pa.device_status(clear=True)
    n0 = pa.launch_count()
    left_out = slots.copy()
    if rope:
        cs = pa.rope_table(maxp, rot).numpy()
        q_out = torch.full((T, hq, d), 7.0, dtype=TORCH_DT[dtype], device="cuda") if hq else None
        if in_place:
            q_out = q
        pa.rope_write_kv_fp8(q if hq else None, k, v, kc, vc, ks, vs, dev(slots), dev(pos), dev(cs), interleaved=il,
                             q_out=q_out)
        assert pa.launch_count() == n0 + (2 if hq else 1)
        assert pa.device_status() == pa.DEV_ERR_SLOT | pa.DEV_ERR_POSITION
        p = np.clip(pos, 0, maxp - 1)
        if hq:
            want = round_to(R.rotate(qkv[:, :hq], cs, p, il), dtype)
            want[pos < 0] = qkv[pos < 0, :hq] if in_place else 7.0
            want[pos >= maxp] = 0.0
            assert np.array_equal(q_out.float().cpu().numpy(), want)
        kt = R.rotate(qkv[:, hq:hq + hkv], cs, p, il)
        left_out[(pos < 0) | (pos >= maxp)] = -1
    else:
        pa.write_kv_fp8(k, v, kc, vc, ks, vs, dev(slots))
        assert pa.launch_count() == n0 + 1 and pa.device_status() == pa.DEV_ERR_SLOT
        kt = qkv[:, hq:hq + hkv]
    # the reference takes a second per three heads: `some` compares a third of them, the first and the last among these
    at = np.unique(np.concatenate([[0, hkv - 1], rng.choice(hkv, hkv // 3, replace=False)])) if some else np.arange(hkv)
    kb, kss, vb, vss = (np.ascontiguousarray(x[:, at]) for x in state)
    R.append_rows(kt[:, at], kb, kss, left_out)
    R.append_rows(qkv[:, hq + hkv:][:, at], vb, vss, left_out)
    pick = torch.from_numpy(at).cuda()
    check_fp8(*(t.view(torch.uint8)[:, pick] if t.element_size() == 1 else t[:, pick] for t in (kc, ks, vc, vs)),
              (kb, kss, vb, vss))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("il", [False, True])
def test_turned_prompts(dtype, d, bs, il):
    require_gpu()
    rng = np.random.default_rng(d + bs + il)
    run(rng, dtype, 5, 32, d, bs, d if bs == 16 else d // 2, il, 5000, 4 if bs == 16 else 2,
        some=il or d == 64)


@pytest.mark.parametrize("hkv,bs,T,heads", [(25, 16, 6300, 4), (33, 16, 2400, 2), (32, 16, 1300, 1)])
def test_head_counts_that_do_not_divide(hkv, bs, T, heads):
    """The last warp of a stretch has fewer heads than the others."""
    require_gpu()
    rng = np.random.default_rng(hkv)
    run(rng, "bf16", 0, hkv, 64, bs, 64, False, T, heads, some=hkv == 32)


@pytest.mark.parametrize("dtype,d", [("fp16", 128), ("bf16", 64)])
def test_without_rotation(dtype, d):
    require_gpu()
    rng = np.random.default_rng(d)
    run(rng, dtype, 0, 32, d, 16, 0, False, 5000, 4, rope=False)


def test_queries_turned_in_place():
    require_gpu()
    rng = np.random.default_rng(7)
    run(rng, "bf16", 9, 32, 128, 16, 96, False, 2600, 2, in_place=True)
