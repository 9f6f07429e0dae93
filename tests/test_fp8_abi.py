"""Host-side refusals of the 8-bit attention and copy calls through the C ABI (no GPU: nothing reaches CUDA)."""
import pytest

import paged_kv_cache_457_b200 as pa
from paged_kv_cache_457_b200 import build_lib


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return pa.load_library()


def call(f, base, **over):
    return f(*{**base, **over}.values())


DECODE = dict(q=16, k=16, v=16, ks=16, vs=16, bt=16, cl=16, scale=0.1, out=16, S=2, hq=4, hkv=2, d=128, bs=16, nb=10, ts=4,
              mcl=40, qs=512, os=512, part=0, dtype=1, ws=None, wsb=0, stream=None)
PREFILL = dict(q=16, k=16, v=16, ks=16, vs=16, bt=16, qst=16, cl=16, scale=0.1, out=16, S=2, N=40, hq=4, hkv=2, d=128,
               bs=16, nb=10, ts=4, mql=32, qs=512, os=512, dtype=1, ws=None, wsb=0, stream=None)
COMMON = ((dict(d=96), -5), (dict(bs=8), -5), (dict(hq=6, hkv=4), -6), (dict(dtype=3), -2), (dict(S=-1), -3),
          (dict(qs=100), -3), (dict(os=100), -3), (dict(q=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
          (dict(out=None), -1), (dict(q=24), -4), (dict(k=24), -4), (dict(ks=18), -4), (dict(bt=18), -4),
          (dict(qs=516), -4), (dict(scale=float("inf")), -3), (dict(scale=float("nan")), -3),
          (dict(nb=1 << 31, hkv=2), -3))


def test_decode_refusals(lib):
    for over, code in COMMON + ((dict(mcl=-1), -3), (dict(nb=0), -3), (dict(ts=0), -3), (dict(part=8), -8),
                                (dict(part=-16), -8), (dict(S=40000), -3)):
        assert call(lib.pa_decode_fp8, DECODE, **over) == code, over
    assert call(lib.pa_decode_fp8, DECODE, S=0) == 0
    assert lib.pa_decode_fp8_workspace_size(2, 4, 2, 96, 16, 40, 0) == 0


def test_prefill_refusals(lib):
    for over, code in COMMON + ((dict(mql=-1), -3), (dict(N=-1), -3), (dict(nb=0), -3), (dict(ts=-1), -3),
                                (dict(S=70000), -3), (dict(qst=None), -1)):
        assert call(lib.pa_prefill_fp8, PREFILL, **over) == code, over
    for none in (dict(S=0), dict(N=0), dict(mql=0)):
        assert call(lib.pa_prefill_fp8, PREFILL, **none) == 0
    assert call(lib.pa_prefill_fp8, PREFILL, ws=None) == -7  # 32 tokens per sequence: the work counter's scratch
    assert lib.pa_prefill_fp8_workspace_size(2, 40, 4, 2, 96, 16, 32) == 0
    assert lib.pa_prefill_fp8_workspace_size(2, 40, 4, 2, 128, 16, 32) == 256


def test_copy_refusals(lib):
    copy = dict(k=16, v=16, ks=16, vs=16, m=16, n=2, hkv=2, d=128, bs=16, nb=10, stream=None)
    for over, code in ((dict(n=-1), -3), (dict(nb=0), -3), (dict(d=80), -5), (dict(bs=64), -5), (dict(ks=None), -1),
                       (dict(m=None), -1), (dict(k=24), -4), (dict(vs=18), -4), (dict(m=20), -4)):
        assert call(lib.pa_copy_blocks_fp8, copy, **over) == code, over
    assert call(lib.pa_copy_blocks_fp8, copy, n=0) == 0
