"""Which kernel a 4-bit product takes, on the CPU: the choice up to the largest
sizes, and that the library has the kernels that some size takes and no others."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from skinny_bf16_decode_amd import LIB_PATH

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path_factory.mktemp("host") / "check_mxfp4_tiles"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall",
           "-Wextra", "-Werror", "-I", os.path.join(ROOT, "skinny_bf16_decode_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "check_mxfp4_tiles.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)

    def run(*args, text=None):
        r = subprocess.run([str(exe), *args], input=text, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.splitlines()

    return run


@pytest.fixture(scope="module")
def reached(check):
    return set(check("reach"))


def test_tiles_cover_the_product_under_sanitizers(check):
    assert check() == ["ok"]


def test_the_library_has_the_kernels_that_are_reached(reached):
    nm = shutil.which("nm")
    if nm is None or not os.path.exists(LIB_PATH):
        pytest.skip("nm or the library is missing")
    listing = subprocess.run([nm, "-C", LIB_PATH], capture_output=True, text=True, check=True).stdout
    built = set()
    for name, args in re.findall(r"__device_stub__(product_\w+)<([^>]*)>", listing):
        a = args.split(", ")
        if name == "product_rows" and len(a) == 6:
            built.add(f"rows {a[0]}x{a[1]} bits {a[2]} x {a[4]} {'once' if a[5] == 'true' else 'again'}")
        elif name != "product_rows" and len(a) == 2:
            built.add(f"tiles {a[0]} bits {8 if name.endswith('8') else 4} {'words' if a[1] == 'true' else 'any'}")
    assert built == reached


def test_gpu_tests_reach_every_kernel(check, reached):
    """The sizes of test_gpu_mxfp4_tiles.py, in the ways in which it lays out powers."""
    from . import test_gpu_mxfp4_tiles as t
    calls = [(m, n, bits, 1) for m, n in t.ROWS for bits in (4, 8)]
    calls += [(m, n, bits, words) for bits, m, n in t.BOTH for words in (0, 1)]
    calls += [(m, n, bits, 1) for bits in (4, 8) for m, n in t.WORDS[bits]]
    names = check("name", text="".join("%d %d %d %d\n" % c for c in calls))
    assert len(names) == len(calls)
    assert all(name.startswith("rows" if c[:2] in t.ROWS else "tiles") for c, name in zip(calls, names))
    assert set(names) == reached


def test_sizes_past_one_launch(check):
    """The sizes of test_gpu_operator_launches.py make more workgroups of 512 threads than one launch may have."""
    tiles = {"4 268436000": "rows 2x2", "8 134218000": "rows 1x1"}
    for name, tokens in (("4 268436000", 32), ("8 134218000", 16)):
        bits, m = map(int, name.split())
        assert check("name", text=f"{m} 7 {bits} 0")[0].startswith(tiles[name]) and m // tokens > 0xFFFFFFFF // 512
    for bits in (4, 8):
        assert check("name", text=f"2 536872000 {bits} 0")[0].startswith("rows 4x1") and 536872000 // 64 > 0xFFFFFFFF // 512
