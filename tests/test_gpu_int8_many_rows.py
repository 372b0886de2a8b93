"""Rows to 8-bit integers, more of them than one launch has workgroups for."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# 64 threads a row with K = 16, 256 with K = 3: past 2^32 threads
@pytest.mark.parametrize("m,k", [(67_300_000, 16), (16_900_000, 3)])
def test_quantize_more_rows_than_a_launch_has(m, k):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import int8
    print("rows", m, k, flush=True)
    x = torch.randn(1000, k, dtype=torch.bfloat16, device="cuda")
    want_q, want_s = int8.quantize_rows(x, torch.empty(1000, k, dtype=torch.int8, device="cuda"),
                                        torch.empty(1000, device="cuda"))
    rows = x.repeat(m // 1000, 1)
    q = torch.full((m, k), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((m,), 7.0, device="cuda")
    int8.quantize_rows(rows, q, scale)
    torch.cuda.synchronize()
    assert bool((q.view(-1, 1000, k) == want_q).all()) and bool((scale.view(-1, 1000) == want_s).all())
