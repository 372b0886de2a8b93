"""The 8-bit product's and linear attention's entry points on the CPU: every
refusal comes before any device call, and the addressing of parts of packed
sequences stays inside the tensors for any starts."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import skinny_bf16_decode_amd as sk
from skinny_bf16_decode_amd import int8, linear_attention as la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
P = 0x10000          # a 16-byte aligned address that is never read


def test_addressing_of_parts_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "check_places"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall",
           "-Wextra", "-Werror", "-I", os.path.join(ROOT, "skinny_bf16_decode_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "check_places.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"{r.stdout}\n{r.stderr}"
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "places ok" in r.stdout, f"{r.stdout}\n{r.stderr}"


@pytest.mark.parametrize("x,kind,m,k,ldx,q,ldq,scale,want", [
    (P, 3, 4, 64, 64, P, 64, P, INVALID),        # no such type
    (P, 0, -1, 64, 64, P, 64, P, INVALID),
    (P, 0, 4, 0, 64, P, 64, P, INVALID),
    (None, 0, 4, 64, 64, P, 64, P, INVALID),
    (P, 0, 4, 64, 64, None, 64, P, INVALID),
    (P, 0, 4, 64, 64, P, 64, None, INVALID),
    (P, 0, 4, 64, 63, P, 64, P, SHAPE),
    (P, 0, 4, 64, 64, P, 63, P, SHAPE),
    (P + 1, 0, 4, 64, 64, P, 64, P, ALIGN),
    (P + 2, 1, 4, 64, 64, P, 64, P, ALIGN),
    (P, 0, 4, 64, 64, P, 64, P + 2, ALIGN),
    (None, 0, 0, 64, 64, None, 64, None, OK),    # no rows: nothing to do
])
def test_quantize_refusals(x, kind, m, k, ldx, q, ldq, scale, want):
    assert sk.load_library().skinny_quantize_rows(x, kind, m, k, ldx, q, ldq, scale, None) == want, sk.last_error()


@pytest.mark.parametrize("w,n,k,ldw,ws,out,want", [
    (None, 16, 64, 64, P, 0, INVALID),
    (P, 16, 64, 64, None, 0, INVALID),
    (P, 0, 64, 64, P, 0, INVALID),
    (P, 16, 0, 64, P, 0, INVALID),
    (P, 16, 64, 64, P, 5, INVALID),
    (P, 16, 72, 72, P, 0, SHAPE),                # K % 16
    (P, 16, 131072, 131072, P, 0, SHAPE),        # 131072 * 128 * 128 does not fit 32 bits
    (P, 16, 64, 63, P, 0, SHAPE),
    (P, 16, 64, 64, P + 1, 0, ALIGN),
])
def test_int8_prepare_refusals(w, n, k, ldw, ws, out, want):
    plan = ctypes.c_void_p(123)
    st = sk.load_library().skinny_int8_prepare(w, n, k, ldw, ws, out, None, ctypes.byref(plan))
    assert st == want and plan.value is None, sk.last_error()
    assert sk.last_error()


def test_int8_prepare_refuses_rows_past_its_counts():
    plan = ctypes.c_void_p(123)
    st = sk.load_library().skinny_int8_prepare(P, 0x7FFFF001, 16, 16, P, 0, None, ctypes.byref(plan))
    assert st == SHAPE and plan.value is None and "at most" in sk.last_error()


def test_int8_null_plans():
    lib = sk.load_library()
    assert lib.skinny_int8_prepare(P, 16, 64, 64, P, 0, None, None) == INVALID
    assert lib.skinny_int8_run(None, P, 64, P, None, 0, P, 16, 4, None) == INVALID
    lib.skinny_int8_destroy(None)


def linear_args(**change):
    a = dict(q=P, k=P, v=P, out=P, log_decay=P, state_in=P, state_out=P, starts=P, slots=P, workspace=None,
             workspace_bytes=0, q_token=64, q_head=32, k_token=64, k_head=32, v_token=64, v_head=32, out_token=64,
             out_head=32, decay_token=2, decay_head=1, in_state_slot=2048, in_state_head=1024, out_state_slot=2048,
             out_state_head=1024, type=0, tokens=3, sequences=3, heads=2, key_heads=2, dk=32, dv=32, pool=4, scale=1.0)
    a.update(change)
    return la._Args(**a)


LINEAR = [
    (dict(type=2), INVALID), (dict(tokens=-1), INVALID), (dict(sequences=-1), INVALID), (dict(pool=-1), INVALID),
    (dict(heads=0), SHAPE), (dict(key_heads=0), SHAPE), (dict(heads=3), SHAPE), (dict(heads=65536), SHAPE),
    (dict(sequences=65536), SHAPE), (dict(dk=0), SHAPE), (dict(dk=12), SHAPE), (dict(dk=264), SHAPE),
    (dict(dv=0), SHAPE), (dict(dv=20), SHAPE), (dict(dv=1032), SHAPE),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(log_decay=None), INVALID), (dict(slots=None, pool=2), SHAPE),
    (dict(q_token=60), SHAPE), (dict(k_head=4), SHAPE), (dict(v_token=-64), SHAPE), (dict(out_token=1 << 24), SHAPE),
    (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(v=P + 4), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(decay_token=-1), SHAPE), (dict(log_decay=P + 2), ALIGN), (dict(slots=P + 1), ALIGN),
    (dict(state_in=P + 4), ALIGN), (dict(state_out=P + 8), ALIGN), (dict(in_state_slot=2), SHAPE),
    (dict(out_state_head=-4), SHAPE),
]


@pytest.mark.parametrize("change,want", LINEAR)
@pytest.mark.parametrize("entry", ["prompt", "step"])
def test_linear_refusals(entry, change, want):
    fn = getattr(sk.load_library(), f"skinny_linear_{entry}")
    assert fn(ctypes.byref(linear_args(**change)), None) == want, (change, sk.last_error())
    assert sk.last_error()


def test_linear_refusals_of_one_entry():
    lib = sk.load_library()
    assert lib.skinny_linear_prompt(None, None) == INVALID
    assert lib.skinny_linear_step(None, None) == INVALID
    assert lib.skinny_linear_step(ctypes.byref(linear_args(tokens=4)), None) == SHAPE
    assert lib.skinny_linear_prompt(ctypes.byref(linear_args(starts=None)), None) == INVALID
    assert lib.skinny_linear_prompt(ctypes.byref(linear_args(starts=P + 2)), None) == ALIGN
    assert lib.skinny_linear_prompt(ctypes.byref(linear_args(sequences=0)), None) == SHAPE
    # nothing to do: no sequence, no token
    none = dict(tokens=0, sequences=0, q=None, k=None, v=None, out=None, log_decay=None)
    assert lib.skinny_linear_prompt(ctypes.byref(linear_args(**none)), None) == OK
    assert lib.skinny_linear_step(ctypes.byref(linear_args(**none)), None) == OK
    # a long prompt needs its workspace, whole and aligned
    need = la.workspace_bytes(100000, 3, 2, 32, 32)
    assert need > 0
    for ws, size, want in ((None, need, INVALID), (P, need - 1, INVALID), (P + 8, need, ALIGN)):
        a = linear_args(tokens=100000, workspace=ws, workspace_bytes=size)
        assert lib.skinny_linear_prompt(ctypes.byref(a), None) == want, (ws, size, sk.last_error())


def test_linear_workspace_sizes():
    assert la.workspace_bytes(1, 1, 12, 128, 128) == 0
    assert la.workspace_bytes(-1, 1, 12, 128, 128) == 0
    assert la.workspace_bytes(100000, 1, 12, 264, 128) == 0      # refused sizes need nothing
    last = 0
    for tokens in (1 << 12, 1 << 15, 1 << 18, 1 << 21):
        b = la.workspace_bytes(tokens, 8, 12, 128, 128)
        assert 0 < b < 1 << 30 and b >= last                     # bounded, whatever the length
        last = b


def test_python_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="on a GPU"):
        int8.quantize_rows(x, q, s)
    with pytest.raises(ValueError, match="BF16, FP16 or fp32"):
        int8.quantize_rows(x.double(), q, s)
    with pytest.raises(ValueError, match="on a GPU"):
        int8.PreparedInt8(q, s)
    h = torch.zeros(4, 2, 32, dtype=torch.bfloat16)
    g, starts = torch.zeros(4, 2), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU|BF16 or FP16"):
        la.prompt(h, h, h, g, torch.empty_like(h), starts)
    with pytest.raises(ValueError, match="BF16 or FP16"):
        la.step(h.float(), h.float(), h.float(), g, h.float())
    with pytest.raises(ValueError, match="starts"):
        la.prompt(h, h, h, g, torch.empty_like(h), starts[:0])
