"""Small 8-bit caches and batches for the tests, and how far the kernels' outputs may be from the 64-bit values."""
from __future__ import annotations

import numpy as np

import fp8_ref as R

HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


class Batch:
    """Sequences of the given context lengths in randomly placed blocks.  Rows that no sequence owns hold NaN bytes
    and scales of blocks in no table are NaN; table entries past a sequence's last block are far out of range."""

    def __init__(self, rng, ctx, hkv, d, bs, spread=1.0, width=None, foreign=False):
        self.ctx = np.asarray(ctx, np.int32)
        self.bs, self.hkv, self.d = bs, hkv, d
        need = -(-self.ctx // bs)
        nb = int(need.sum()) + 2
        free = rng.permutation(nb)
        self.tables = np.full((len(ctx), width or max(1, int(need.max(initial=1)))), 2 ** 31 - 1, np.int32)
        live = np.zeros(nb, int)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = free[at:at + n]
            for i in range(n):
                live[free[at + i]] = min(bs, self.ctx[s] - i * bs)
            at += n
        self.pools = []
        for _ in range(2):
            x = rng.standard_normal((nb, hkv, bs, d)).astype(np.float32)
            x *= np.exp2(np.rint(rng.uniform(-np.log2(spread), np.log2(spread), (nb, hkv, 1, 1)))).astype(np.float32)
            b, s = R.quantise_pool(x)
            if foreign:  # scales that are no powers of two
                s = (s * rng.uniform(0.5, 1.0, s.shape)).astype(np.float32)
            b[np.broadcast_to((np.arange(bs)[None] >= live[:, None])[:, None, :, None], b.shape)] = 0x7F
            s[live == 0] = np.nan
            self.pools += [b, s]

    def values(self):
        """K and V in float64; dead rows zero."""
        out = []
        for b, s in ((self.pools[0], self.pools[1]), (self.pools[2], self.pools[3])):
            out.append(np.nan_to_num(R.values(b, s), nan=0.0))
        return out


def tolerance(out, mean_abs, dots, keys, d, dtype, v_max, p_half_step=2.0 ** -11, p_floor=2.0 ** -32, kv_half_step=0.0):
    """Elementwise bound of |kernel - exact|; `keys`: context length of each row [N], `v_max`: the largest value the
    cache's bytes can stand for (448 times the largest scale).

    A weight w is off by a relative e: half a step of the type it is rounded to (p_half_step); the score's fp32 dot of
    d products and its scaling, (d + 8) 2^-24 of sum |scale q k| in nats, taken twice for the running maximum's share;
    what rounding K to the storage type moves it (kv_half_step of the same sum); 2^-20 for the exponential's and
    logarithm's approximations.  Numerator and normaliser see the same w, so the output moves by at most
    e (sum w |v| + |out|); their fp32 sums over L keys add L 2^-24 of each, rounded V kv_half_step of sum w |v|.
    Weights too small for their type's normal numbers are off by p_floor of the largest: L p_floor v_max.  Then half a
    step of the output's type (2^-25 below fp16's normal range)."""
    L = np.asarray(keys, np.float64)[:, None, None]
    e = p_half_step + (2 * (d + 8) * 2.0 ** -24 + 2 * kv_half_step) * dots[:, :, None] + 2.0 ** -20 + 2 * L * 2.0 ** -24
    err = e * (mean_abs + np.abs(out)) + kv_half_step * mean_abs + L * p_floor * v_max
    return err + HALF_STEP[dtype] * (np.abs(out) + err) + 2.0 ** -25
