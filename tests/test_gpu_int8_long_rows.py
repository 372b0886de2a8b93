"""Rows to 8-bit integers of the longest length: a thread's index behind such a row's end passes 2^31."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_quantize_the_longest_row():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import int8
    k = 2147483647
    print("row", k, flush=True)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(1, k, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    x[0, k - 1] = 60.0                      # the row's largest, its last
    q, scale = torch.full((1, k + 1), 77, dtype=torch.int8, device="cuda"), torch.zeros(1, device="cuda")
    int8.quantize_rows(x, q[:, :k], scale)
    torch.cuda.synchronize()
    top = torch.full((1,), 60.0, device="cuda")
    assert torch.equal(scale, top / torch.full_like(top, 127.0)) and int(q[0, k]) == 77 and int(q[0, k - 1]) == 127
    inverse = torch.full_like(top, 127.0) / top
    for a in range(0, k, 1 << 27):
        c = slice(a, min(a + (1 << 27), k))
        assert torch.equal(q[0, c], torch.round(x[0, c].float() * inverse).to(torch.int8)), a
    del x, q
    torch.cuda.empty_cache()
