"""The built kernels' stores of more than 8 bytes a lane: no data register of one
is written by the instruction after it.

A vector store reads its data over several cycles.  The compiler leaves the
next instruction free to overwrite the data of a buffer store whose offset is in
a scalar register; on gfx950 such a store wrote the next instruction's result in
its first data register, from lanes 12 to 15 of every 16.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from skinny_bf16_decode_amd import LIB_PATH

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
STORE = re.compile(r"\s(buffer|global|flat|scratch)_store_dwordx[34]\s+(.*?)\s*//")
WRITE = re.compile(r"\s(v_\w+)\s+(v\[\d+:\d+\]|v\d+)[,\s]")


def registers(text):
    m = re.fullmatch(r"v\[(\d+):(\d+)\]", text)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"v(\d+)", text)
    return {int(m[1])} if m else set()


def overwritten(listing):
    """(stores seen, [(function, store, next instruction)] of those whose data the next instruction writes)."""
    found, stores, function = [], 0, ""
    for line, after in zip(listing, listing[1:]):
        if line.startswith("<"):
            function = line
        m = STORE.search(line)
        if not m:
            continue
        stores += 1
        operands = [x.strip() for x in m[2].split(",")]
        data = registers(operands[0 if m[1] == "buffer" else 1].split()[0])
        w = WRITE.search(after)
        if w and data & registers(w[2]):
            found.append((function, line.split("//")[0].strip(), after.split("//")[0].strip()))
    return stores, found


def test_the_search_finds_an_overwritten_store():
    store = "\tbuffer_store_dwordx4 v[114:117], v118, s[20:23], s3 offen // 0: 0"
    for after, count in (("\tv_mul_f32_e32 v114, v122, v153 // 8: 0", 1), ("\tv_mfma_f32_16x16x32_f16 v[112:115], v[0:3], v[4:7], 0 // 8: 0", 1),
                         ("\tv_mul_f32_e32 v118, v114, v153 // 8: 0", 0), ("\ts_nop 0 // 8: 0", 0)):
        assert len(overwritten([store, after])[1]) == count, after
    assert len(overwritten(["\tglobal_store_dwordx4 v[0:1], v[4:7], off // 0: 0", "\tv_mov_b32_e32 v5, 0 // 8: 0"])[1]) == 1


def test_no_wide_store_is_overwritten(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    shutil.copy(LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    stores = 0
    for name in sorted(os.listdir(tmp_path)):
        if "gfx950" not in name:
            continue
        r = subprocess.run([OBJDUMP, "-d", "--no-leading-addr", name], cwd=tmp_path, check=True, capture_output=True,
                           text=True)
        seen, found = overwritten(r.stdout.splitlines())
        stores += seen
        assert not found, (name, found)
    assert stores > 0
