"""The index-checked build is the release build with the checks in, and nothing else: what its tests find holds for both."""
from paged_kv_cache_457_b200 import build_lib


def test_the_debug_build_differs_in_its_checks_alone():
    release, debug = build_lib.command("out.so"), build_lib.command("out.so", debug=True)
    assert [x for x in debug if x != "-DPA_DEBUG"] == release
    assert debug.count("-DPA_DEBUG") == 1
