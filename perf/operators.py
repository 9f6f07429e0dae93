"""What the 8-bit cache path and the rotating append are measured on: cases, inputs, plain forms and exact values.

Four operators of a serving step over the paged cache:

* ``append``     -- queries and keys turned by their position, keys and values appended to a 16-bit paged cache;
* ``append_fp8`` -- the same into a cache held in 8 bits (e4m3) with one scale for each block of tokens and head;
* ``decode_fp8`` -- attention of one new token per sequence over such a cache;
* ``prefill_fp8`` -- causal attention of several new tokens per sequence over such a cache.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and this framework's calls; ``exact``
gives the same outputs in 64 bits.  Lengths follow from the case alone, values and block placement from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
MAX_POSITION = 32768  # positions the angle table covers


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a very small step: four sequences of a small model, one token each; launch latency is all there is
        dict(name="append tiny step", op="append", dtype="fp16", hq=8, hkv=8, d=64, bs=16, rot=64, interleaved=False,
             seqs=4, lo=1, hi=200, new=1, pad=0, spread=1),
        # one decode step of a large continuous batch with grouped heads, padded to a fixed batch for graph replay
        dict(name="append 250 sequences", op="append", dtype="bf16", hq=32, hkv=8, d=128, bs=16, rot=128,
             interleaved=False, seqs=250, lo=16, hi=8192, new=1, pad=6, spread=2),
        # a chunked-prefill step: 32 sequences bring 512 tokens each behind cached prefixes
        dict(name="append prompt chunks", op="append", dtype="bf16", hq=32, hkv=8, d=128, bs=16, rot=128,
             interleaved=False, seqs=32, lo=0, hi=3584, new=512, pad=0, spread=3),
        # the decode step's append into the 8-bit cache: most blocks are partly filled, some scales have to grow
        dict(name="append fp8 250 sequences", op="append_fp8", dtype="bf16", hq=32, hkv=8, d=128, bs=16, rot=128,
             interleaved=False, seqs=250, lo=16, hi=8192, new=1, pad=6, spread=4),
        # whole prompts of a model with one kv head per query head: the largest append
        dict(name="append fp8 prompts", op="append_fp8", dtype="fp16", hq=32, hkv=32, d=128, bs=16, rot=128,
             interleaved=False, seqs=16, lo=0, hi=0, new=1283, pad=0, spread=5),
        # four short sequences of a small model
        dict(name="decode fp8 tiny", op="decode_fp8", dtype="fp16", hq=8, hkv=8, d=64, bs=16, seqs=4, lo=1, hi=200,
             dist="uniform", spread=6),
        # a decode batch without grouped heads
        dict(name="decode fp8 64 sequences", op="decode_fp8", dtype="fp16", hq=32, hkv=32, d=128, bs=16, seqs=64,
             lo=128, hi=2048, dist="uniform", spread=7),
        # a large continuous batch with grouped heads and a long tail of lengths
        dict(name="decode fp8 grouped heads", op="decode_fp8", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=256,
             lo=16, hi=8192, dist="lognormal", spread=8),
        # few sequences with long contexts: the work has to be split along the tokens
        dict(name="decode fp8 long context", op="decode_fp8", dtype="bf16", hq=32, hkv=32, d=128, bs=32, seqs=8,
             lo=16384, hi=32768, dist="uniform", spread=9),
        # a few tokens per sequence behind a context (a drafted continuation, ragged chunk ends)
        dict(name="prefill fp8 few tokens", op="prefill_fp8", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=8,
             lo=100, hi=2000, new_lo=1, new_hi=9, spread=10),
        # whole short prompts, odd lengths
        dict(name="prefill fp8 prompts", op="prefill_fp8", dtype="fp16", hq=32, hkv=32, d=128, bs=16, seqs=16,
             lo=0, hi=0, new_lo=130, new_hi=1100, spread=11),
        # the chunked-prefill step with grouped heads
        dict(name="prefill fp8 chunks", op="prefill_fp8", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=32,
             lo=0, hi=3584, new_lo=512, new_hi=512, spread=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "append_fp8", "decode_fp8", "decode_fp8", "prefill_fp8"])
    hq, hkv = rng.choice([(8, 8), (32, 32), (32, 8), (16, 8), (12, 4), (32, 4), (16, 1), (7, 1), (5, 5)])
    d = rng.choice([64, 128])
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), hq=hq, hkv=hkv, d=d, bs=rng.choice([16, 32]),
             spread=rng.randrange(1 << 20))
    if op in ("append", "append_fp8"):
        c["rot"] = rng.choice([d, d, d // 2, 16])
        c["interleaved"] = rng.random() < 0.3
        if rng.random() < 0.5:  # a decode step
            c.update(seqs=_log_int(rng, 1, 512), lo=1, hi=_log_int(rng, 16, 8192), new=1, pad=rng.randrange(8))
        else:  # prompt chunks
            seqs = _log_int(rng, 1, 32)
            c.update(seqs=seqs, lo=0, hi=_log_int(rng, 16, 4000), new=_log_int(rng, 2, 16384 // seqs),
                     pad=rng.randrange(8))
    elif op == "decode_fp8":
        seqs = _log_int(rng, 1, 256)
        # tokens in all: at most what the largest listed case reads, and the plain form's products stay in 32-bit sizes
        most = min(196608 * 32 * 128 // (hkv * d), 400_000_000 // (hq * d))
        hi = _log_int(rng, 16, max(17, min(32768, most // seqs)))
        c.update(seqs=seqs, lo=rng.choice([0, 1, max(1, hi // 8)]), hi=hi, dist="uniform")
    else:
        seqs = _log_int(rng, 1, 32)
        new_hi = _log_int(rng, 1, 600)
        most = 2 ** 31 // (seqs * hq * new_hi)
        hi = _log_int(rng, 1, max(2, min(3584, most - new_hi)))
        c.update(seqs=seqs, lo=0, hi=hi, new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi)
    return c


def _lens(c):
    """Tokens of each sequence before the new ones (append, prefill) or in all (decode)."""
    r = random.Random(c["spread"])
    if c.get("dist") == "lognormal":
        return [min(c["hi"], max(c["lo"], int(round(math.exp(r.gauss(math.log(512.0), 1.0)))))) for _ in range(c["seqs"])]
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return lens if any(lens) else lens[:-1] + [c["hi"]]


def _new(c):
    r = random.Random(c["spread"] + 7)
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    return new if any(new) else new[:-1] + [c["new_hi"]]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(g, dtype, *shape):
    """Activations: normal, a few channels of each head larger than the others, as keys of trained models have."""
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    gain = 1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.05).float()
    return (x * gain).to(DTYPES[dtype])


def _pow2_scale(amax):
    """The smallest power of two s (from 2^-64 on) with amax <= 448 s: bytes re-scaled by such steps keep their bits."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875)).clamp(min=-64).masked_fill(amax == 0, -64).int()
    return ((e + 127) << 23).view(torch.float32)


def _pool(g, c, live):
    """Blocks of random rows in 8 bits with their scales; `live`: int tensor [blocks], rows of each block in use.
    Dead rows hold the NaN pattern."""
    nb, hkv, bs, d = live.numel(), c["hkv"], c["bs"], c["d"]
    out = torch.empty((nb, hkv, bs, d), dtype=F8, device="cuda")
    scale = torch.empty((nb, hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (hkv * bs * d))
    for a in range(0, nb, step):
        x = torch.randn((min(step, nb - a), hkv, bs, d), generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-1, 2, (x.shape[0], hkv, 1, 1), generator=g, device="cuda").float())
        dead = (torch.arange(bs, device="cuda") >= live[a:a + step, None])[:, None, :, None]
        x.masked_fill_(dead, 0.0)
        s = _pow2_scale(x.abs().amax((2, 3)))
        b = (x / s[:, :, None, None]).to(F8).view(torch.uint8)
        out[a:a + step] = b.masked_fill(dead, 0x7F).view(F8)
        scale[a:a + step] = s
    return out, scale


def _place(g, lens, bs):
    """A table of randomly placed blocks for sequences of these lengths, and each block's rows in use."""
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    width = max(1, max(need))
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    n = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    owned = col[None] < n[:, None]
    first = torch.cumsum(n, 0) - n
    tables = torch.where(owned, perm[(first[:, None] + col[None]).clamp(max=nb - 1)], -1).int().contiguous()
    length = torch.tensor(lens, device="cuda")
    rows = (length[:, None] - col[None] * bs).clamp(0, bs)
    live = torch.zeros(nb, dtype=torch.long, device="cuda")
    live[tables[owned].long()] = rows[owned]
    return tables, live


def _angles(rot):
    """cos and sin of position * 10000^(-2i / rot), computed in 64 bits, stored as [position][cos... sin...]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _append_tokens(c):
    """(sequence, position) counts: per sequence the position of its first new token, and its new tokens."""
    if c["new"] == 1:
        return [max(0, n - 1) for n in _lens(c)], [1] * c["seqs"]
    r = random.Random(c["spread"] + 7)
    return _lens(c), [r.randint(max(1, c["new"] // 2), c["new"]) if c["lo"] == c["hi"] else c["new"] for _ in range(c["seqs"])]


def _prepare_append(c, seed):
    g = _gen(seed)
    first, count = _append_tokens(c)
    bs = c["bs"]
    # the pool holds the blocks this step writes: from the block of each sequence's first new token on
    tables, live = _place(g, [f % bs + n for f, n in zip(first, count)], bs)
    f, n = torch.tensor(first, device="cuda"), torch.tensor(count, device="cuda")
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), n)
    at = torch.arange(seq.numel(), device="cuda") - (torch.cumsum(n, 0) - n)[seq]
    inside = f[seq] % bs + at
    slots = tables[seq, inside // bs].long() * bs + inside % bs
    positions = f[seq] + at
    if c["pad"]:
        tail = torch.full((c["pad"],), -1, dtype=torch.long, device="cuda")
        slots, positions = torch.cat([slots, tail]), torch.cat([positions, tail])
    tokens = slots.numel()
    # one projection's output holds q, k and v side by side, as a fused projection leaves them
    qkv = _rows(g, c["dtype"], tokens, c["hq"] + 2 * c["hkv"], c["d"])
    q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], 1)
    s = dict(c=c, q=q, k=k, v=v, slots=slots, positions=positions, cos_sin=_angles(c["rot"]),
             q_out=torch.zeros((tokens, c["hq"], c["d"]), dtype=DTYPES[c["dtype"]], device="cuda"))
    if c["op"] == "append":
        shape = (live.numel(), c["hkv"], bs, c["d"])
        s["k_cache"], s["v_cache"] = _rows(g, c["dtype"], *shape), _rows(g, c["dtype"], *shape)
    else:
        old = torch.zeros_like(live)  # rows that earlier steps wrote
        old[tables[:, 0].long()] = f % bs
        s["k_cache"], s["k_scale"] = _pool(g, c, old)
        s["v_cache"], s["v_scale"] = _pool(g, c, old)
    return s


def _prepare_attention(c, seed):
    g = _gen(seed)
    lens = _lens(c)
    new = [1] * c["seqs"]
    if c["op"] == "prefill_fp8":
        new = _new(c)
        lens = [a + b for a, b in zip(lens, new)]
    tables, live = _place(g, lens, c["bs"])
    s = dict(c=c, tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), longest=max(lens),
             scale=1.0 / math.sqrt(c["d"]))
    s["k_cache"], s["k_scale"] = _pool(g, c, live)
    s["v_cache"], s["v_scale"] = _pool(g, c, live)
    s["q"] = torch.randn((sum(new), c["hq"], c["d"]), generator=g, device="cuda").to(DTYPES[c["dtype"]])
    if c["op"] == "prefill_fp8":
        s["new"], s["most_new"] = new, max(new)
        s["query_start"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
    else:
        s["total"] = sum(lens)
    return s


def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"].startswith("append") else _prepare_attention(case, seed)


# ---------------------------------------------------------------- plain forms
def _turn(x, angle, rot, interleaved):
    """x [T, H, d] in 32 bits turned by the angles [T, rot] of its tokens; dims from rot on pass."""
    c, s = angle[:, None, :rot // 2], angle[:, None, rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    c = s["c"]
    bs = c["bs"]
    there = s["positions"] >= 0
    angle = s["cos_sin"][s["positions"].clamp(min=0)]
    q = _turn(s["q"].float(), angle, c["rot"], c["interleaved"]).to(s["q"].dtype)
    s["q_out"].copy_(torch.where(there[:, None, None], q, s["q_out"]))
    k = _turn(s["k"].float(), angle, c["rot"], c["interleaved"])
    v = s["v"].float()
    writes = s["slots"].numel() - c["pad"]  # padding comes last
    block, row = s["slots"][:writes] // bs, s["slots"][:writes] % bs
    if c["op"] == "append":
        s["k_cache"][block, :, row] = k[:writes].to(s["k"].dtype)
        s["v_cache"][block, :, row] = s["v"][:writes]
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    started = torch.zeros(s["k_cache"].shape[0], device="cuda").index_add_(0, block, (row == 0).float()) > 0
    for x, cache, scale in ((k[:writes], s["k_cache"], s["k_scale"]), (v[:writes], s["v_cache"], s["v_scale"])):
        fine = torch.where(x.isfinite(), x, 0.0)
        amax = torch.zeros_like(scale).index_reduce_(0, block, fine.abs().amax(-1), "amax")
        touched = torch.zeros_like(started)
        touched[block] = True
        wanted = _pow2_scale(amax)
        grown = torch.where(touched[:, None], torch.where(started[:, None], wanted, torch.maximum(scale, wanted)), scale)
        kept = torch.where(started[:, None], 1.0, scale / grown)  # rows of earlier steps in units of the new scale
        cache.copy_(torch.where((kept == 1.0)[:, :, None, None], cache.float(), cache.float() * kept[:, :, None, None]).to(F8))
        scale.copy_(grown)
        cache.view(torch.uint8)[block, :, row] = (x / grown[block][:, :, None]).clamp(-448.0, 448.0).to(F8).view(torch.uint8)
    return [s["q_out"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]]


def _plain_decode(s):
    c = s["c"]
    bs, group = c["bs"], c["hq"] // c["hkv"]
    n = s["lens"].long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["total"])
    at = torch.arange(s["total"], device="cuda") - (torch.cumsum(n, 0) - n)[seq]
    block, row = s["tables"][seq, at // bs].long(), at % bs
    k = s["k_cache"].view(torch.uint8)[block, :, row].view(F8).float() * s["k_scale"][block][:, :, None]
    z = (s["q"].float().view(-1, c["hkv"], group, c["d"])[seq] * k[:, :, None]).sum(-1) * s["scale"]
    top = torch.full((n.numel(),) + z.shape[1:], -math.inf, device="cuda").index_reduce_(0, seq, z, "amax")
    w = torch.exp(z - top[seq])
    total = torch.zeros_like(top).index_add_(0, seq, w)
    v = s["v_cache"].view(torch.uint8)[block, :, row].view(F8).float() * s["v_scale"][block][:, :, None]
    out = torch.zeros(top.shape + (c["d"],), device="cuda").index_add_(0, seq, w[..., None] * v[:, :, None])
    out = out / torch.where(total > 0, total, 1.0)[..., None]
    return out.view(-1, c["hq"], c["d"]).to(s["q"].dtype)


def _plain_prefill(s):
    c = s["c"]
    bs, group, d = c["bs"], c["hq"] // c["hkv"], c["d"]
    start, lens = s["query_start"].long(), s["lens"].long()
    new = start[1:] - start[:-1]
    t = torch.arange(s["most_new"], device="cuda")
    j = torch.arange(s["longest"], device="cuda")
    there = j[None] < lens[:, None]
    block = torch.where(there, s["tables"][:, (j // bs).clamp(max=s["tables"].shape[1] - 1)].long(), 0)
    row = (j % bs)[None].expand_as(block)
    hide = ~there[:, :, None, None]
    k = (s["k_cache"].view(torch.uint8)[block, :, row].view(F8).float() * s["k_scale"][block][..., None]).masked_fill(hide, 0.0)
    v = (s["v_cache"].view(torch.uint8)[block, :, row].view(F8).float() * s["v_scale"][block][..., None]).masked_fill(hide, 0.0)
    at = (start[:-1, None] + t[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(len(lens), len(t), c["hkv"], group, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    z = (q @ k.permute(0, 2, 3, 1)).view(len(lens), c["hkv"], group, len(t), len(j)) * s["scale"]
    seen = j[None, None] <= ((lens - new)[:, None] + t[None])[:, :, None]
    z = z.masked_fill(~(seen & there[:, None])[:, None, None], -math.inf)
    w = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
    total = w.sum(-1, keepdim=True)
    o = (w.flatten(2, 3) @ v.permute(0, 2, 1, 3)).view(len(lens), c["hkv"], group, len(t), d)
    o = (o / torch.where(total > 0, total, 1.0)).permute(0, 3, 1, 2, 4).reshape(len(lens), len(t), c["hq"], d)
    tokens = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(start[1:], tokens, right=True)
    return o[seq, tokens - start[seq]].to(s["q"].dtype)


def _own(s):
    import paged_kv_cache_457_b200 as pa
    op = s["c"]["op"]
    if op == "append":
        pa.rope_write_kv(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["cos_sin"],
                         interleaved=s["c"]["interleaved"], q_out=s["q_out"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if op == "append_fp8":
        pa.rope_write_kv_fp8(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"],
                             s["positions"], s["cos_sin"], interleaved=s["c"]["interleaved"], q_out=s["q_out"])
        return [s["q_out"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]]
    if op == "decode_fp8":
        return pa.decode_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["tables"], s["lens"],
                             s["scale"], max_context_len=s["longest"])
    return pa.prefill_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["tables"],
                          s["query_start"], s["lens"], s["scale"], s["most_new"])


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    if op.startswith("append"):
        return _plain_append(state)
    return _plain_decode(state) if op == "decode_fp8" else _plain_prefill(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(c):
    hq, hkv, d, bs = c["hq"], c["hkv"], c["d"], c["bs"]
    if c["op"].startswith("append"):
        first, count = _append_tokens(c)
        t = sum(count)
        elem = 2 if c["op"] == "append" else 1
        # q in and out, k and v in, rows out, angles, slots and positions; scales of the blocks written, read and written
        b = t * (2 * hq * d * 2 + 2 * hkv * d * (2 + elem) + c["rot"] * 4 + 16)
        if elem == 1:
            b += sum(-(-(f % bs + n) // bs) for f, n in zip(first, count)) * hkv * 2 * 8
        return dict(bytes=b, flops=t * (hq + hkv) * c["rot"] * 3)
    lens, new = _lens(c), [1] * c["seqs"]
    if c["op"] == "prefill_fp8":
        new = _new(c)
        lens = [a + b for a, b in zip(lens, new)]
    pairs = sum(n * (n + 1) // 2 + n * (m - n) for m, n in zip(lens, new)) if c["op"] == "prefill_fp8" else sum(lens)
    live = [m for m, n in zip(lens, new) if n]
    blocks = sum(-(-m // bs) for m in live)
    b = sum(live) * hkv * d * 2 + blocks * (hkv * 8 + 4) + sum(new) * hq * d * 4 + 4 * c["seqs"]
    return dict(bytes=b, flops=4 * pairs * hq * d)


# ---------------------------------------------------------------- exact values, in 64 bits
def _e4m3(x):
    """x in 64 bits rounded to the nearest of e4m3's values, ties to the even one, at most 448 in size."""
    a = x.abs().clamp(max=448.0)
    unit = _two_to(torch.frexp(a.clamp(min=2.0 ** -6))[1].long() - 4)  # values from 2^(e-1) on are 2^(e-4) apart
    return torch.sign(x) * (torch.round(a / unit) * unit).clamp(max=448.0)


def _two_to(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_append(s):
    c = s["c"]
    rot, bs = c["rot"], c["bs"]
    keep = (s["positions"] >= 0).nonzero()[:, 0]
    angle = s["cos_sin"].double()[s["positions"][keep]]
    # a pair of dims as one complex number, turned by multiplication with cos + i sin
    unit = torch.complex(angle[:, :rot // 2], angle[:, rot // 2:])[:, None]

    def turned(x):
        x = x[keep].double()
        y = x.clone()
        even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., even], x[..., odd]) * unit
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    q = s["q_out"].double()
    q[keep] = turned(s["q"])
    slots = s["slots"][keep]
    out = [q]
    for x, name in ((turned(s["k"]), "k"), (s["v"][keep].double(), "v")):
        if c["op"] == "append":
            pool = s[name + "_cache"].double().transpose(1, 2).flatten(0, 1).clone()
            pool[slots] = x
            out.append(pool.view(-1, bs, c["hkv"], c["d"]).transpose(1, 2).contiguous())
            continue
        pool = s[name + "_cache"].double().transpose(1, 2).flatten(0, 1).clone()  # [slot, head, d]
        scale = s[name + "_scale"].double().clone()
        order = torch.argsort(slots)
        blocks, n = torch.unique_consecutive(slots[order] // bs, return_counts=True)
        top = torch.segment_reduce(x[order].abs().amax(-1), "max", lengths=n)
        fresh = (slots[order] % bs)[torch.cumsum(n, 0) - n] == 0
        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).long()
        e = torch.where(_two_to(e - 1) * 448.0 >= top, e - 1, torch.where(_two_to(e) * 448.0 < top, e + 1, e))
        want = _two_to(e.clamp(min=-64))
        was = scale[blocks]
        now = torch.where(fresh[:, None], want, torch.maximum(was, want))
        rows = pool.view(-1, bs, c["hkv"], c["d"])[blocks]
        move = (~fresh[:, None] & (now > was))[:, None, :, None]
        again = _e4m3(rows * (was / now)[:, None, :, None])
        pool.view(-1, bs, c["hkv"], c["d"])[blocks] = torch.where(move, again, rows)
        scale[blocks] = now
        pool[slots] = _e4m3(x / scale[slots // bs][..., None])
        out += [pool.view(-1, bs, c["hkv"], c["d"]).transpose(1, 2).contiguous(), scale]
    return out


def _exact_attention(s):
    c = s["c"]
    bs, group, d = c["bs"], c["hq"] // c["hkv"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    first = s["query_start"].tolist() if "query_start" in s else list(range(len(lens) + 1))
    for i, m in enumerate(lens):
        a, b = first[i], first[i + 1]
        if m == 0 or a == b:
            continue
        ids = s["tables"][i, :-(-m // bs)].long()

        def context(name):
            x = s[name + "_cache"][ids].double() * s[name + "_scale"][ids].double()[:, :, None, None]
            return x.transpose(0, 1).reshape(c["hkv"], -1, d)[:, :m]

        k, v = context("k"), context("v")
        seen = torch.arange(m, device="cuda")[None] <= torch.arange(m - (b - a), m, device="cuda")[:, None]
        for h in range(c["hkv"]):
            q = s["q"][a:b, h * group:(h + 1) * group].double().transpose(0, 1)
            z = (q @ k[h].T * s["scale"]).masked_fill(~seen, -math.inf)
            out[a:b, h * group:(h + 1) * group] = (torch.softmax(z, -1) @ v[h]).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"].startswith("append") else _exact_attention(s)
