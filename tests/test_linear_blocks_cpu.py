"""The order in which linear attention's workgroups take the parts of packed sequences, on the CPU."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_order_of_parts_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "check_blocks"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall",
           "-Wextra", "-Werror", "-I", os.path.join(ROOT, "skinny_bf16_decode_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "check_blocks.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_token_counts_past_the_parts_arithmetic_are_refused():
    import skinny_bf16_decode_amd as sk
    from skinny_bf16_decode_amd import linear_attention as la
    p = 0x10000                 # a 16-byte aligned address that is never read
    a = la._Args(q=p, k=p, v=p, out=p, log_decay=p, starts=p, q_token=64, k_token=64, v_token=64, out_token=64, type=0,
                 tokens=0x7FFFF001, sequences=1, heads=1, key_heads=1, dk=32, dv=32, pool=0, scale=1.0)
    assert sk.load_library().skinny_linear_prompt(ctypes.byref(a), None) == 2 and "at most" in sk.last_error()
    assert la.workspace_bytes(0x7FFFF001, 1, 1, 32, 32) == 0
