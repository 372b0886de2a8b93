"""How norms and joins deal rows to threads, on the CPU: sizes up to the longest row."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path_factory.mktemp("host") / "check_norm_shape"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall",
           "-Wextra", "-Werror", "-I", os.path.join(ROOT, "skinny_bf16_decode_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "check_norm_shape.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    return str(exe)


def test_every_element_has_a_place_under_sanitizers(check):
    r = subprocess.run([check], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


KINDS = {None: 0, "int8": 1, "mx4": 2, "mx8": 3}


def test_gpu_tests_reach_every_kernel(check):
    """The calls of test_gpu_norms_kernels.py, by the kernels that norms.hip has for each type."""
    from . import test_gpu_norms_kernels as t
    types = range(3)                        # skinny_type: BF16, fp32, FP16
    calls = []
    for x in types:
        for m, k, off, q in t.NORMS:
            calls.append(("norm", x, None, f"norm {m} {k} {x} {int(not off and k % 8 == 0)} {KINDS[q]}"))
        for m, k in t.STREAMED:
            calls.append(("norm", x, None, f"norm {m} {k} {x} 1 {KINDS['int8']}"))
        for r in types:
            for m, k, off, q, token in t.JOINS:
                calls.append(("join", x, r, f"join {m} {k} {x} {r} {int(not off and k % 8 == 0)} {KINDS[q]} {int(token)}"))
            for m, k in t.JOINED:
                calls.append(("join", x, r, f"join {m} {k} {x} {r} 1 {KINDS['int8']} 0"))
    r = subprocess.run([check, "name"], input="\n".join(c[3] for c in calls), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    names = r.stdout.splitlines()
    assert len(names) == len(calls)
    kernels = [f"{octets} {mode}" for mode, many in (("vectors", (1, 2, 4, 0)), ("elements", (1, 0)), ("strided", (1, 2, 0)))
               for octets in many]
    want = set()
    for x in types:
        want |= {("norm", x, None, f"norm_kernel {n}") for n in kernels}
        want |= {("norm", x, None, f"norm_stream {c} 1") for c in (1, 2, 3)}
        if x != 1:
            want.add(("norm", x, None, "norm_stream 1 4"))
        for r in types:
            want |= {("join", x, r, f"join_kernel {n}") for n in kernels}
            want.add(("join", x, r, f"join_stream 1 {1 if 1 in (x, r) else 2}"))
    assert {(*c[:3], name) for c, name in zip(calls, names)} == want
