"""The workspace of linear attention's prompts, on the CPU: one for the largest prompt serves all smaller ones."""
from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

from skinny_bf16_decode_amd import linear_attention as la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sizes_and_states_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "check_shape"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall",
           "-Wextra", "-Werror", "-I", os.path.join(ROOT, "skinny_bf16_decode_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "check_shape.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_a_larger_prompt_needs_no_less():
    rng = random.Random(5)
    for _ in range(20000):
        heads, dk, dv = rng.choice([1, 2, 12, 40]), 8 * rng.randint(1, 32), 8 * rng.randint(1, 64)
        tokens, b = int(2 ** rng.uniform(0, 19)), int(2 ** rng.uniform(0, 11))
        more, further = tokens + rng.randint(0, 40000), b + rng.randint(0, 30)
        assert la.workspace_bytes(tokens, b, heads, dk, dv) <= la.workspace_bytes(more, further, heads, dk, dv), (
            tokens, b, more, further, heads, dk, dv)


def test_many_short_sequences():
    """Only sequences that are cut have states in it: two for every 256 tokens, not one for every sequence."""
    heads, dk, dv = 12, 128, 128
    state = heads * dk * dv * 4
    assert la.workspace_bytes(200000, 2000, heads, dk, dv) <= 2 * (200000 // 256) * (state + heads * 8)
    assert la.workspace_bytes(100000, 512, heads, dk, dv) <= 2 * (100000 // 256) * (state + heads * 8)
    assert la.workspace_bytes(100000, 65535, heads, dk, dv) <= 2 * (100000 // 256) * (state + heads * 8)


def test_more_workgroups_than_a_launch_has_are_refused():
    """2^32 threads in one launch would run a part of them without an error."""
    import ctypes

    import skinny_bf16_decode_amd as sk
    p = 0x10000                 # a 16-byte aligned address that is never read
    for heads, key_heads, dk, dv in ((300, 300, 32, 32), (256, 1, 128, 128), (32, 16, 64, 1024)):
        a = la._Args(q=p, k=p, v=p, out=p, log_decay=p, starts=p, q_token=64, k_token=64, v_token=64, out_token=64,
                     type=0, tokens=65535, sequences=65535, heads=heads, key_heads=key_heads, dk=dk, dv=dv, pool=0,
                     scale=1.0, workspace=p, workspace_bytes=1 << 50)
        assert sk.load_library().skinny_linear_prompt(ctypes.byref(a), None) == 2, (heads, dv)
        assert "too many" in sk.last_error()
