"""The 8-bit split kernel's chunks, walked on the host with the cut that the kernel compiles."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_457_b200", "csrc")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("chunks") / "walk")
    cxx = shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, "-o", out, os.path.join(HERE, "chunk_walk.cpp")], check=True)

    def run(*args):
        return [int(x) for x in subprocess.run([out, *map(str, args)], check=True, capture_output=True, text=True).stdout.split()]
    return run


@pytest.mark.parametrize("cut", [0, 1, 2, 3, 16])
@pytest.mark.parametrize("total", [1, 2, 3, 39, 40, 41, 400, 1777, 3552, 3553, 20001])
def test_the_arithmetic_meets_every_tile_under_its_own_name(walk, total, cut):
    for warps in (4, 20, 1776):
        room = max(1, -(-total // cut)) if cut else warps * 4 + 1  # what the host plans for
        wrong, left, used, c = walk(total, warps, cut, room)
        assert (wrong, left, used) == (0, 0, total)
        assert -(-total // c) <= room
        if cut >= 2:
            assert c == cut
