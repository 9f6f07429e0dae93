"""The plain reference of the 8-bit cache against torch's e4m3 type, and its append against hand-worked cases."""
import numpy as np
import torch

import fp8_ref as R


def test_e4m3_table_and_rounding_match_torch():
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(R.E4M3)) and np.array_equal(t[~np.isnan(t)], R.E4M3[~np.isnan(t)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.integers(-4, 3, 20000), R.E4M3[:0x7F],
                        (R.E4M3[:0x7E] + R.E4M3[1:0x7F]) / 2, -(R.E4M3[:0x7E] + R.E4M3[1:0x7F]) / 2]).astype(np.float32)
    x = np.clip(x, -448, 448)
    assert np.array_equal(R.e4m3_bytes(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_pow2_scale_is_the_smallest_that_holds_the_rows():
    for amax, want in ((448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (1.0, 2.0 ** -8),
                       (0.0, 2.0 ** -64)):
        assert R.pow2_scale(amax) == want


def test_append_grows_the_scale_and_keeps_older_rows():
    cache, scale = np.full((2, 1, 16, 64), 0x7F, np.uint8), np.zeros((2, 1), np.float32)
    x = np.zeros((3, 1, 64), np.float32)
    x[0], x[1], x[2] = 3.0, 100.0, 0.25
    R.append_rows(x[:1], cache, scale, np.array([16]))  # row 0 of block 1
    assert scale[1, 0] == 2.0 ** -7 and np.all(R.values(cache, scale)[1, 0, 0] == 3.0)
    R.append_rows(x[1:], cache, scale, np.array([17, 18]))
    assert scale[1, 0] == 0.25
    got = R.values(cache, scale)[1, 0, :3]
    # 100 / 0.25 = 400 lies midway between e4m3's 384 and 416: to the even one
    assert np.all(got[0] == 3.0) and np.all(got[1] == 96.0) and np.all(got[2] == 0.25)
    R.append_rows(x[2:], cache, scale, np.array([16]))  # the block starts anew: a small scale again
    assert scale[1, 0] == 2.0 ** -10
