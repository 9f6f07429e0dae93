"""The 8-bit kernels' window of a block table row, driven on the host through the code that the kernels compile."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_457_b200", "csrc")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("window") / "walk")
    cxx = shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, "-o", out, os.path.join(HERE, "table_window.cpp")], check=True)

    def run(*args):
        return [int(x) for x in subprocess.run([out, *map(str, args)], check=True, capture_output=True, text=True).stdout.split()]
    return run


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("new,per,longest", [(9, 2, 500), (4, 1, 300), (24, 8, 200), (24, 2, 2100), (1, 1, 3000)])
def test_every_entry_a_tile_needs_is_held(walk, bs, new, per, longest):
    for seed in range(4):
        missing, _, loads = walk(seed, bs, new, per, longest)
        assert missing == 0 and loads > 0


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("new,per,longest", [(9, 2, 500), (24, 8, 200), (1, 1, 3000), (1, 1, 15)])
def test_no_entry_behind_a_groups_last_block_is_read(walk, bs, new, per, longest):
    """The row may be the last of a table that ends with that entry."""
    for seed in range(4):
        _, past, loads = walk(seed, bs, new, per, longest)
        assert past == 0 and loads > 0
