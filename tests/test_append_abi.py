"""Host-side refusals of the rotating and 8-bit appends through the C ABI (no GPU: nothing reaches CUDA)."""
import pytest

import paged_kv_cache_457_b200 as pa
from paged_kv_cache_457_b200 import build_lib


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return pa.load_library()


ROPE = dict(q=16, k=16, v=16, qo=16, kc=16, vc=16, sm=16, pos=16, cs=16, T=4, hq=4, hkv=2, d=128, rot=128, il=0, bs=16,
            nb=10, maxp=64, qs=512, ks=256, vs=256, qos=512, dtype=1, stream=None)


def rope(lib, **over):
    return lib.pa_rope_write_kv(*{**ROPE, **over}.values())


def rope8(lib, **over):
    a = {**ROPE, "ksc": 16, "vsc": 16, **over}
    order = ["q", "k", "v", "qo", "kc", "vc", "ksc", "vsc", "sm", "pos", "cs", "T", "hq", "hkv", "d", "rot", "il", "bs",
             "nb", "maxp", "qs", "ks", "vs", "qos", "dtype", "stream"]
    return lib.pa_rope_write_kv_fp8(*[a[n] for n in order])


@pytest.mark.parametrize("call", [rope, rope8])
def test_rope_refusals(lib, call):
    for over, code in ((dict(T=-1), -3), (dict(hkv=0), -3), (dict(nb=0), -3), (dict(hq=-1), -3), (dict(dtype=3), -2),
                       (dict(d=96), -5), (dict(bs=8), -5), (dict(rot=0), -5), (dict(rot=24), -5), (dict(rot=144), -5),
                       (dict(maxp=0), -3), (dict(hkv=1 << 20), -3), (dict(k=None), -1), (dict(sm=None), -1),
                       (dict(pos=None), -1), (dict(cs=None), -1), (dict(q=None), -1), (dict(qo=None), -1),
                       (dict(ks=128), -3), (dict(vs=128), -3), (dict(qs=256), -3), (dict(qos=256), -3),
                       (dict(qs=1024), -3),  # q_out is q with another stride
                       (dict(q=24), -4), (dict(k=24), -4), (dict(kc=24), -4), (dict(qs=516), -4), (dict(ks=260), -4),
                       (dict(pos=20), -4), (dict(sm=20), -4), (dict(cs=24), -4)):
        assert call(lib, **over) == code, over
    assert call(lib, T=0) == 0
    assert call(lib, T=0, q=None, hq=0) == 0


def test_fp8_refusals(lib):
    assert rope8(lib, ksc=None) == -1
    assert rope8(lib, vsc=18) == -4
    w = lib.pa_write_kv_fp8
    ok = [16, 16, 16, 16, 16, 16, 16, 4, 2, 128, 16, 10, 256, 256, 1, None]
    for i, x, code in ((0, None, -1), (4, None, -1), (5, 18, -4), (7, -1, -3), (9, 80, -5), (10, 64, -5), (11, 0, -3),
                       (12, 100, -3), (14, 0, -2)):
        a = list(ok)
        a[i] = x
        assert w(*a) == code, (i, x)
    ok[7] = 0
    assert w(*ok) == 0


def test_rope_table_is_computed_in_64_bits():
    import math
    t = pa.rope_table(40000, 64)
    assert t.shape == (40000, 64) and str(t.dtype) == "torch.float32"
    for p, i in ((0, 0), (39999, 0), (39999, 1), (12345, 31)):
        a = p * 10000.0 ** (-2 * i / 64)
        # float32 rounding of a value of size <= 1: half a step is 2^-25; the rest is float64's
        assert abs(t[p, i].item() - math.cos(a)) <= 2.0 ** -25 + 1e-10
        assert abs(t[p, 32 + i].item() - math.sin(a)) <= 2.0 ** -25 + 1e-10


def test_binding_refuses_cpu_tensors_and_non_tensors():
    import torch
    f8 = torch.zeros((2, 1, 16, 64), dtype=torch.float8_e4m3fn)
    h, s = torch.zeros((2, 1, 16, 64), dtype=torch.float16), torch.ones((2, 1))
    x, i = torch.zeros((3, 1, 64), dtype=torch.float16), torch.zeros(3, dtype=torch.int64)
    t, c = torch.zeros((3, 1), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    cs = pa.rope_table(4, 64)
    for call in (lambda: pa.rope_write_kv(x, x, x, h, h, i, i, cs), lambda: pa.write_kv_fp8(x, x, f8, f8, s, s, i),
                 lambda: pa.rope_write_kv_fp8(x, x, x, f8, f8, s, s, i, i, cs),
                 lambda: pa.decode_fp8(x, f8, f8, s, s, t, c, 0.1, 1),
                 lambda: pa.prefill_fp8(x, f8, f8, s, s, t, torch.zeros(4, dtype=torch.int32), c, 0.1, 1),
                 lambda: pa.copy_blocks_fp8(f8, f8, s, s, torch.zeros((1, 2), dtype=torch.int64)),
                 lambda: pa.decode_fp8(x, None, f8, s, s, t, c, 0.1, 1),
                 lambda: pa.write_kv_fp8(x, [1], f8, f8, s, s, i)):
        with pytest.raises(pa.PagedAttentionError):
            call()
