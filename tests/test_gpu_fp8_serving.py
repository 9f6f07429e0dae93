"""The 8-bit cache as a server uses it: pages and scales moved by copies, and a run of steps planned by the block
manager (chunked prompts, fork, copy-on-write, decode, swap out and in), each step's outputs against the 64-bit
reference on what the cache then holds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref as R
import paged_kv_cache_457_b200 as pa
from fp8_cases import HALF_STEP, tolerance
from gpu_util import TORCH_DT, require_gpu

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def random_pool(rng, nb, hkv, bs, d):
    k, v = (torch.from_numpy(rng.integers(0, 256, (nb, hkv, bs, d), dtype=np.uint8)) for _ in range(2))
    ks, vs = (torch.from_numpy(rng.standard_normal((nb, hkv)).astype(np.float32)) for _ in range(2))
    return [k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs]


def same(a, b):
    return torch.equal(a.view(torch.uint8).cpu(), b.view(torch.uint8).cpu())


@pytest.mark.parametrize("hkv,bs,d", [(1, 16, 64), (3, 32, 64), (8, 16, 128), (40, 16, 64)])
@pytest.mark.parametrize("n", [0, 1, 9])
def test_copy_blocks_moves_bytes_and_scales(hkv, bs, d, n):
    require_gpu()
    rng = np.random.default_rng(hkv + bs + n)
    nb = 40
    host = random_pool(rng, nb, hkv, bs, d)
    pool = [t.cuda() for t in host]
    ids = rng.permutation(nb)[:2 * n].reshape(n, 2).astype(np.int64)
    if n == 9:
        ids[2, 0], ids[5, 1] = -1, -1
    pa.copy_blocks_fp8(*pool, dev(ids))
    for t, h in zip(pool, host):
        want = h.clone()
        for a, b in ids:
            if a >= 0 and b >= 0:
                want.view(torch.uint8 if t.element_size() == 1 else torch.float32)[b] = \
                    h.view(torch.uint8 if t.element_size() == 1 else torch.float32)[a]
        assert same(t, want)
    assert pa.device_status() == 0


def test_swap_blocks_through_pinned_memory_and_flags():
    require_gpu()
    rng = np.random.default_rng(3)
    hkv, bs, d, nb, hb = 5, 16, 128, 12, 6
    host = random_pool(rng, nb, hkv, bs, d)
    pool = [t.cuda() for t in host]
    pinned = [torch.zeros((hb,) + tuple(t.shape[1:]), dtype=t.dtype).pin_memory() for t in host]
    out = dev(np.array([[3, 0], [7, 5], [1, 2], [nb, 1], [2, hb]], np.int64))
    pa.swap_blocks_fp8(*pool, *pinned, out)
    assert pa.device_status() == pa.DEV_ERR_BLOCK_ID
    back = dev(np.array([[0, 10], [5, 11], [2, 9]], np.int64))
    pa.swap_blocks_fp8(*pinned, *pool, back)
    assert pa.device_status() == 0
    for t, h in zip(pool, host):
        t, h = t.cpu().view(torch.uint8).reshape(nb, -1), h.view(torch.uint8).reshape(nb, -1)
        for a, b in ((3, 10), (7, 11), (1, 9)):
            assert torch.equal(t[b], h[a])
        assert torch.equal(t[:9], h[:9])


def test_copy_refusals():
    require_gpu()
    rng = np.random.default_rng(4)
    pool = [t.cuda() for t in random_pool(rng, 4, 2, 16, 64)]
    m = dev(np.array([[0, 1]], np.int64))
    n0 = pa.launch_count()
    for bad in (lambda: pa.copy_blocks_fp8(*pool, m.int()), lambda: pa.copy_blocks_fp8(*pool[:3], pool[3].half(), m),
                lambda: pa.copy_blocks_fp8(*pool, m.cpu()), lambda: pa.copy_blocks_fp8(pool[0].half(), *pool[1:], m),
                lambda: pa.swap_blocks_fp8(*pool, *[t[:, :1].contiguous() for t in pool], m),
                lambda: pa.swap_blocks_fp8(*pool, *[t.cpu() for t in pool], m)):
        with pytest.raises(pa.PagedAttentionError):
            bad()
    assert pa.launch_count() == n0


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("fp16", 32)])
def test_server_run(dtype, bs):
    """Two prompts prefilled in chunks, one forked, both decoded with copy-on-write, one swapped out and back."""
    require_gpu()
    rng = np.random.default_rng(bs)
    hq, hkv, d, nb, hb, width = 8, 2, 128, 48, 24, 24
    scale, table = d ** -0.5, pa.rope_table(512, d, device="cuda")
    kc, vc = (torch.zeros((nb, hkv, bs, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, hkv), device="cuda") for _ in range(2))
    pinned = [torch.zeros((hb,) + tuple(t.shape[1:]), dtype=t.dtype).pin_memory() for t in (kc, vc, ks, vs)]
    bm = pa.BlockManager(bs, nb, hb)
    rows = {}  # sequence -> the float64 K and V it has appended

    def cos_sin64():
        return table.double().cpu().numpy()

    def step(seqs, new, plan, decode):
        """Append and attend; returns nothing, checks outputs and what the cache holds."""
        T = int(sum(new))
        qkv = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)).to(TORCH_DT[dtype])
        first = [bm.num_tokens(s) - n for s, n in zip(seqs, new)]
        pos = np.concatenate([np.arange(f, f + n) for f, n in zip(first, new)]).astype(np.int64)
        q, k, v = qkv.cuda().split([hq, hkv, hkv], 1)
        if len(plan.copy_pairs):
            pa.copy_blocks_fp8(kc, vc, ks, vs, dev(np.asarray(plan.copy_pairs, np.int64).reshape(-1, 2)))
        q = pa.rope_write_kv_fp8(q, k, v, kc, vc, ks, vs, dev(plan.slot_mapping), dev(pos), table)
        ctx = np.asarray(plan.context_lens)
        if decode:
            out = pa.decode_fp8(q, kc, vc, ks, vs, dev(plan.block_tables), dev(ctx), scale, max_context_len=int(ctx.max()))
        else:
            out = pa.prefill_fp8(q, kc, vc, ks, vs, dev(plan.block_tables), dev(plan.query_start), dev(ctx), scale,
                                 int(max(new)))
        assert pa.device_status() == 0
        pools = [R.values(t.view(torch.uint8).cpu().numpy(), s.cpu().numpy()) for t, s in ((kc, ks), (vc, vs))]
        ref, mean_abs, dots = R.attention(q.double().cpu().numpy(), *pools, np.asarray(plan.block_tables), ctx, scale,
                                          new=new, bounds=True)
        tol = tolerance(ref, mean_abs, dots, np.repeat(ctx, new), d, dtype, 448.0 * float(vs.max()), HALF_STEP[dtype],
                        2.0 ** -25)
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)
        # what the cache holds: every appended row, off by e4m3's half step 2^-4 and, where the block's scale grew,
        # by another (subnormal bytes: half of 2^-9 scales, twice)
        x = qkv.double().numpy()
        turned = R.rotate(x[:, hq:hq + hkv], cos_sin64(), pos, False)
        at = 0
        for s, n in zip(seqs, new):
            rows.setdefault(s, []).append((turned[at:at + n], x[at:at + n, hq + hkv:]))
            at += n
        for i, s in enumerate(seqs):
            L = int(ctx[i])
            ids = np.asarray(plan.block_tables)[i, :-(-L // bs)]
            for which, (pool, sc) in enumerate(((pools[0], ks), (pools[1], vs))):
                held = pool[ids].transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:L]
                unit = np.repeat(sc.cpu().numpy()[ids], bs, 0)[:L, :, None]
                want = np.concatenate([r[which] for r in rows[s]])
                assert want.shape[0] == L
                assert np.all(np.abs(held - want) <= 2 * (2.0 ** -4 * np.abs(want) + 2.0 ** -10 * unit))

    new = [70, 33]
    for s, n in enumerate(new):
        bm.add_sequence(s, 0)
    done = [0, 0]
    while any(d_ < n for d_, n in zip(done, new)):
        chunk = [min(29, n - d_) for d_, n in zip(done, new)]
        plan = bm.build_prefill_step([0, 1], chunk, table_stride=width)
        step([0, 1], chunk, plan, False)
        done = [a + c for a, c in zip(done, chunk)]
    bm.fork(0, 2)
    rows[2] = list(rows[0])
    for _ in range(2 * bs + 3):
        plan = bm.build_decode_step([0, 1, 2], table_stride=width)
        step([0, 1, 2], [1, 1, 1], plan, True)
    pairs = np.asarray(bm.swap_out([1]), np.int64).reshape(-1, 2)
    pa.swap_blocks_fp8(kc, vc, ks, vs, *pinned, dev(pairs))
    step([0, 2], [1, 1], bm.build_decode_step([0, 2], table_stride=width), True)
    pairs = np.asarray(bm.swap_in([1]), np.int64).reshape(-1, 2)
    pa.swap_blocks_fp8(*pinned, kc, vc, ks, vs, dev(pairs))
    step([0, 1, 2], [1, 1, 1], bm.build_decode_step([0, 1, 2], table_stride=width), True)
    # a mixed step: drafted continuations of different lengths
    step([0, 1, 2], [4, 1, 6], bm.build_prefill_step([0, 1, 2], [4, 1, 6], table_stride=width), False)
